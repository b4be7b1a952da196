"""Attention over the quantised cache where its numerics are at their edges:
queries that are not finite, values beyond fp16, keys of few large channels; and
where its work is cut: row blocks inside a token, requests of many lengths.
Tolerances are those of the attention's own tests.
"""
import threading

import numpy as np
import pytest
import torch

from oracle import kv
from tests.test_gpu_attn_kv import Setup
from tests.test_gpu_kv_cache import dev, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("ctx", [40, 2900])
@pytest.mark.parametrize("elem,D,G,n", [(kv.I8, 128, 4, 1), (kv.I4, 128, 4, 4), (kv.I8, 64, 4, 8), (kv.I8, 128, 4, 10),
                                        (kv.I4, 64, 4, 40)])
def test_queries_that_are_not_numbers(us, elem, D, G, n, ctx, value):
    """exp of a NaN score, and infinite scores' differences, are NaN: so are that row's outputs, and no
    other's, whether a segment is one CTA's or many CTAs'."""
    s = Setup(us, elem, D, 1, G, 64, [ctx], [n], 31)
    words, grids = s.tree()
    clean, at = s.run(words), (n // 2, 1)
    codes = np.array([kv.unpack(s.ref.k[s.ref.at(0, p)[0], 0, s.ref.at(0, p)[1]], elem)[5] for p in range(ctx)])
    assert (codes > 0).any() and (codes < 0).any()              # one score is +inf, whichever sign the query has
    s.Q[at][5] = value
    got = s.run(words)
    assert np.isnan(got[at]).all()
    got[at], s.Q[at][5] = clean[at], 0
    keep = clean[at].copy()
    want, mag, big = kv.attend(s.ref, 0, s.Q, ctx, grids[0], s.scale)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -24 + mag * (2 * 2.0 ** -11 + 2 * (D + 8) * 2.0 ** -24 * big[..., None])
    tol[at] = np.inf
    assert np.array_equal(keep, got[at]) and (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("elem,scale,code", [(kv.I8, 512.0, -128), (kv.I8, 1024.0, 127), (kv.I4, 8192.0, -8), (kv.I4, 16384.0, 7)])
@pytest.mark.parametrize("D,G,n", [(128, 4, 4), (64, 4, 8), (64, 1, 6), (128, 4, 10), (64, 8, 64), (128, 8, 32)])
def test_unseen_entries_of_large_values(us, elem, scale, code, D, G, n):
    """A drafted entry whose values are beyond fp16's leaves the rows that do not see it as they are."""
    s = Setup(us, elem, D, 1, G, 16, [90], [n], 33)
    words, grids = s.tree()
    words[:] &= ~np.int64(1 << (n - 1)) if n < 64 else np.int64(2 ** 63 - 1)
    for g in grids[0]:
        g[n - 1] = 0
    page, slot = s.ref.at(0, 90 + n - 1)
    s.ref.v[page, :, slot] = kv.pack(np.full((1, D), code), elem)
    s.ref.scale[page, :, slot, 1] = scale
    s.C = us.KVCache(elem, D, s.C.k, dev(s.ref.v), dev(s.ref.scale), s.C.page_table)
    s.check(s.run(words), grids)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,G,n", [(128, 4, 1), (64, 4, 1), (128, 4, 4), (64, 8, 4), (128, 4, 16), (128, 8, 32)])
def test_keys_of_few_large_channels(us, elem, D, G, n):
    """Four channels set the keys' scales and the other codes are 0 or 1; queries are large where all codes
    are 0.  Scores are small sums of the products that are left: nothing else may enter their rounding."""
    s = Setup(us, elem, D, 1, G, 16, [60], [n], 32)
    rng, r, q = s.rng, s.ref, kv.QMAX[elem]
    large = rng.choice(np.arange(0, D, 2), 4, replace=False)
    free = np.setdiff1d(np.arange(0, D, 2), large)
    codes = np.zeros((*r.k.shape[:3], D), np.int64)
    codes[..., large] = rng.choice([-q, q], codes[..., large].shape)
    np.put_along_axis(codes, rng.choice(free, (*codes.shape[:3], 1)), 1, -1)
    r.k[:] = kv.pack(codes, elem)
    fin = np.isfinite(r.scale[..., 0].astype(np.float32))
    r.scale[..., 0][fin] = 5 / s.scale                          # scores of about 200
    s.Q[:] = 40 + 2 * rng.standard_normal(s.Q.shape)
    s.Q[..., 1::2] = 12000 + 1000 * rng.standard_normal(s.Q[..., 1::2].shape)
    s.Q[..., large] = 0
    s.C = us.KVCache(elem, D, dev(r.k), s.C.v, dev(r.scale), s.C.page_table)
    words, grids = s.tree()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,G,n", [(128, 4, 1), (128, 4, 4), (64, 4, 8), (128, 4, 10), (64, 8, 64)])
def test_largest_values_stay_finite(us, elem, D, G, n):
    """V of +-65504 throughout: its entries stand for a little more, the outputs do not."""
    s = Setup(us, elem, D, 1, G, 16, [300], [n], 34)
    x = s.rng.choice([-65504.0, 65504.0], D)
    c, sc = kv.quantise(x, elem)
    fin = np.isfinite(s.ref.scale[..., 1].astype(np.float32))
    s.ref.v[:] = kv.pack(c, elem)
    s.ref.scale[..., 1][fin] = sc
    s.C = us.KVCache(elem, D, s.C.k, dev(s.ref.v), dev(s.ref.scale), s.C.page_table)
    got = s.run(s.tree()[0])
    # sums of equal values: within the weights' rounding of +-65532 (65520), and at most 65504
    assert (np.sign(got) == np.sign(x)).all() and (np.abs(got) <= 65504).all()
    assert (np.abs(got) >= 65504 * (1 - 3 * 2.0 ** -11)).all()


@pytest.mark.parametrize("G,n", [(4, 2), (4, 33)])
def test_calls_of_several_threads(us, G, n):
    """Host threads with a stream and a workspace each."""
    s = Setup(us, kv.I8, 64, 1, G, 16, [700], [n], 37)
    words, grids = s.tree()
    want = s.run(words)
    q, m, off, pos = dev(s.Q), dev(words), dev(offsets(s.n)), dev(np.array(s.ctx, np.int32))
    outs = [torch.zeros(n, s.Hq, 64, dtype=torch.float16, device="cuda") for _ in range(4)]
    sets = [(torch.cuda.Stream(), us.workspace_attn_kv(s.C, s.Hq, n), o) for o in outs]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(sets)), []

    def work(stream, ws, o):
        try:
            start.wait(timeout=60)
            for _ in range(20):
                us.us_attn_kv(s.C, q, off, pos, m, n, s.scale, o, ws, stream=stream)
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and us.us_get_last_device_status() == us.US_OK
    assert all(np.array_equal(o.cpu().numpy().astype(np.float64), want) for o in outs)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,G,ctx,n", [
    (128, 1, 5, [0, 37], [110, 9]), (64, 1, 7, [128, 1], [90, 40]), (128, 1, 3, [127], [190]), (64, 2, 5, [0], [60]),
    (128, 1, 5, [70, 3], [5, 6]), (64, 1, 3, [16, 250], [10, 7]), (128, 1, 8, [100], [100]), (64, 1, 7, [0], [37])])
def test_chains_of_several_row_blocks(us, elem, D, Hkv, G, ctx, n):
    """Query heads that do not divide a block's rows: blocks begin inside a token, on both kernels."""
    s = Setup(us, elem, D, Hkv, G, 32, ctx, n, 35)
    words, grids = s.chain()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,G,tree", [(128, 4, False), (64, 8, True), (128, 7, True)])
def test_long_requests_beside_single_tokens(us, elem, D, G, tree):
    n = [1, 50, 1, 0, 1, 64, 2] if tree else [1, 1, 150, 0, 1, 3, 1]
    s = Setup(us, elem, D, 2 if G == 4 else 1, G, 16, [300, 20, 0, 9, 128, 65, 700], n, 36)
    words, grids = s.tree() if tree else s.chain()
    s.check(s.run(words, pad=8), grids)


@pytest.mark.parametrize("number", [-2 ** 31, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("B,ctx,n,G,bad", [(1024, 511, 1, 4, 3), (2, 90, 16, 4, 1)])
def test_any_bad_page_number_is_recorded(us, B, ctx, n, G, bad, number):
    """Whichever tile of its share a CTA meets it in; the request's other positions are attended to."""
    s = Setup(us, kv.I4, 64, 1, G, 16, [ctx] * B, [n] * B, 38)
    words, grids = s.chain()
    s.C.page_table[bad, 0] = number
    o = torch.zeros(s.T, s.Hq, 64, dtype=torch.float16, device="cuda")
    us.us_attn_kv(s.C, dev(s.Q), dev(offsets(s.n)), dev(np.array(s.ctx, np.int32)), None, n, s.scale, o,
                  us.workspace_attn_kv(s.C, s.Hq, n))
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    got = o.cpu().numpy().astype(np.float64)
    s.check(got, grids, only={0, 1, B - 1} - {bad})
    s.ref.table = s.ref.table.copy()
    s.ref.table[bad, :-1], s.ref.table[bad, -1] = s.ref.table[bad, 1:], -1
    s.ctx[bad] = ctx - 16                                       # positions 0..15 are not attended to
    s.check(got, grids, only={bad})
