"""Norm and rotation on the GPU against the plain reference in 64 bits.

Tolerance.  In fp32: the sum of D squares in sums of 8 and then a tree is off by at most
(8 + 5) 2^-24 of itself, half of which reaches 1 / sqrt, whose own error is 2 ulp; the
products add five roundings: 2^-20 of the value.  The angle: 2^-33 turns, the fraction's
fp32 rounding 2^-25 of half a turn, sincospi 2 ulp: below 2^-22 radians, of a value's
partner.  fp16: 2^-11 of the result, or half the smallest step.
|err| <= 2^-11 |y| + 2^-25 + 2^-20 (|a| + |b|), a, b the pair before its rotation."""
import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_gpu_kv_cache import dev, offsets

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def i32(v):
    return dev(np.array(v, np.int32))


def freqs(R, base=10000.0):
    return base ** (-2.0 * np.arange(R // 2) / max(R, 1))


def rope(us, R, style, eps=EPS):
    return us.Rope(style, us.rope_freq(torch.from_numpy(freqs(R))).cuda(), eps)


def values(rng, T, H, D):
    return (rng.standard_normal((T, H, D)) * np.exp(2 * rng.standard_normal((T, H, 1)))).astype(np.float16)


def check(got, x, w, p, R, style, eps=EPS):
    n = lat.norm(x, w, eps)
    want = lat.rotate(n, p, freqs(R), style == 1)
    size = np.abs(lat.rotate(np.abs(n), np.zeros(len(x)), freqs(R), False))     # |a| + |b| of each value's pair
    half, part = R // 2, np.abs(n)
    if R:
        other = part.copy()
        if style == 1:
            other[..., 0:R:2], other[..., 1:R:2] = part[..., 1:R:2], part[..., 0:R:2]
        else:
            other[..., :half], other[..., half:R] = part[..., half:R], part[..., :half]
        other[..., R:] = 0
        size = part + other
    err = np.abs(got.astype(np.float64) - want)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -20 * size
    assert (err <= tol).all(), f"{np.max(err / tol):.2f} times the tolerance"


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("D,R,Hq,Hkv,n,ctx,normed", [
    (128, 128, 32, 8, [1] * 16, [1000 - 3 * b for b in range(16)], True),
    (128, 64, 5, 1, [3, 0, 40, 1], [0, 7, 130000, 2 ** 30 - 50], True),
    (64, 64, 4, 4, [33], [5], False),
    (64, 32, 7, 1, [1, 2, 3], [9, 99, 999], True),
    (96, 48, 3, 3, [17], [11], True),
    (256, 256, 2, 1, [9, 30], [2, 70000], True),
    (192, 64, 16, 1, [5], [40], True),
    (16, 16, 9, 2, [21], [1], True),
    (8, 0, 1, 1, [4], [0], True),
    (128, 0, 8, 8, [12, 13], [3, 4], True),
    (128, 128, 1, 1, [700], [123456], True),
])
def test_against_the_reference(us, style, D, R, Hq, Hkv, n, ctx, normed):
    rng = np.random.default_rng(D + R)
    T = sum(n)
    x = values(rng, T, Hq + 2 * Hkv, D)
    x[0] = 0                                                     # a token of zeros
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float16) if normed else None for _ in range(2)]
    wd = [None if u is None else dev(u) for u in w]
    fused = torch.full((T + 2, (Hq + 2 * Hkv) * D + 16), 9.0, dtype=torch.float16, device="cuda")
    fused[:T, :-16] = dev(x).reshape(T, -1)
    heads = fused[:T, :-16].unflatten(1, (Hq + 2 * Hkv, D))
    q, k = heads[:, :Hq], heads[:, Hq:Hq + Hkv]
    qo, ko = (torch.full((T + 1, H, D), 7.0, dtype=torch.float16, device="cuda") for H in (Hq, Hkv))
    r, off, pos = rope(us, R, style), dev(offsets(n)), i32(ctx)
    us.us_norm_rope(r, q, wd[0], qo[:T], k, wd[1], ko[:T], off, pos, None, max(n) + 5)
    assert us.us_get_last_device_status() == us.US_OK
    p = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, n)])
    check(qo[:T].cpu().numpy(), x[:, :Hq], w[0], p, R, style)
    check(ko[:T].cpu().numpy(), x[:, Hq:Hq + Hkv], w[1], p, R, style)
    assert (qo[T:] == 7).all() and (ko[T:] == 7).all()            # rows behind the last token stay
    # by their depths, in place, one at a time
    depth = rng.integers(0, 9, T)
    dd = i32(depth)
    us.us_norm_rope(r, q, wd[0], q, None, None, None, off, pos, dd, max(n))
    us.us_norm_rope(r, None, None, None, k, wd[1], k, off, pos, dd, max(n))
    pd = np.concatenate([np.full(m, c) for c, m in zip(ctx, n)]) + depth
    check(q.cpu().numpy(), x[:, :Hq], w[0], pd, R, style)
    check(k.cpu().numpy(), x[:, Hq:Hq + Hkv], w[1], pd, R, style)
    assert np.array_equal(heads[:, Hq + Hkv:].cpu().numpy(), x[:, Hq + Hkv:])          # the value heads beside them stay
    assert (fused[T:] == 9).all() and (fused[:T, -16:] == 9).all()


def test_part_of_a_head_in_place(us):
    """The last 64 values of 192-wide heads, the way latent queries are turned."""
    rng = np.random.default_rng(3)
    x = values(rng, 11, 6, 192)
    xd = dev(x)
    part = xd[..., 128:]
    us.us_norm_rope(rope(us, 64, 1), part, None, part, None, None, None, i32([0, 4, 11]), i32([100, 0]), None, 7)
    assert us.us_get_last_device_status() == us.US_OK
    p = np.concatenate((np.arange(100, 104), np.arange(7)))
    got = xd.cpu().numpy()
    check(got[..., 128:], x[..., 128:], None, p, 64, 1)
    assert np.array_equal(got[..., :128], x[..., :128])


def test_rows_with_infinities_and_nan_stay_among_themselves(us):
    rng = np.random.default_rng(4)
    x = values(rng, 6, 3, 64)
    x[2, 1, 5], x[4, 0, 0] = np.inf, np.nan
    w = np.ones(64, np.float16)
    out = torch.zeros(6, 3, 64, dtype=torch.float16, device="cuda")
    us.us_norm_rope(rope(us, 64, 0), dev(x), dev(w), out, None, None, None, i32([0, 6]), i32([0]), None, 6)
    got = out.cpu().numpy()
    assert np.isnan(got[4, 0]).all() and np.isnan(got[2, 1]).any()
    got[4, 0], x[4, 0], got[2, 1], x[2, 1] = 0, 0, 0, 0
    check(got, x, w, np.arange(6), 64, 0)


def test_bad_offsets_skip_the_request(us):
    rng = np.random.default_rng(5)
    x = values(rng, 8, 2, 64)
    out = torch.full((8, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    us.us_norm_rope(rope(us, 64, 0), dev(x), None, out, None, None, None, i32([0, 3, 2, 8]), i32([0, 0, 1]), None, 6)
    assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
    check(out[:2].cpu().numpy(), x[:2], None, np.arange(2), 64, 0)
    # row 2 is the first request's third and the last one's first: either may come last
    one, other = [lat.rotate(lat.norm(x[2:3], None, EPS), np.array([p]), freqs(64), False) for p in (2, 1)]
    first = np.abs(out[2:3].cpu().numpy() - one).max() < np.abs(out[2:3].cpu().numpy() - other).max()
    check(out[2:3].cpu().numpy(), x[2:3], None, np.array([2 if first else 1]), 64, 0)
    check(out[3:].cpu().numpy(), x[3:], None, 2 + np.arange(5), 64, 0)


@pytest.mark.parametrize("elem", ["I8", "I4"])
@pytest.mark.parametrize("D,R,style,Hq,Hkv,page,n,ctx,depths", [
    (128, 128, 0, 32, 8, 16, [1] * 16, list(range(16)), False),
    (64, 32, 1, 7, 1, 16, [13, 0, 30], [3, 5, 250], True),
    (128, 64, 1, 2, 2, 64, [300], [60], False),
    (64, 64, 0, 0, 4, 32, [40, 2], [1, 31], False),
    (128, 128, 0, 40, 8, 16, [70], [0], True),
])
def test_append_is_norm_and_rotation_then_write(us, elem, D, R, style, Hq, Hkv, page, n, ctx, depths):
    """The same bits, in the cache and out of it."""
    rng = np.random.default_rng(D + Hq)
    T, e = sum(n), getattr(us, "US_" + elem)
    x = values(rng, T, Hq + 2 * Hkv, D)
    x[T // 2, -1, 3], x[T // 2, Hq, 1] = np.inf, np.nan
    wq, wk = (dev((1 + 0.3 * rng.standard_normal(D)).astype(np.float16)) for _ in range(2))
    xd = dev(x)
    q, k, v = (xd[:, :Hq] if Hq else None), xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    need = [-(-max(c + m, 1) // page) for c, m in zip(ctx, n)]
    ids = rng.permutation(sum(need) + 2)
    table = np.full((len(n), max(need)), -1, np.int32)
    for b, m in enumerate(need):
        table[b, :m] = ids[sum(need[:b]):sum(need[:b + 1])]
    r, off, pos = rope(us, R, style), dev(offsets(n)), i32(ctx)
    depth = i32(rng.integers(0, 12, T)) if depths else None
    empty = lambda H: torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda") if H else None  # noqa: E731
    A, B = (us.kv_cache(e, D, Hkv, page, len(ids), dev(table)) for _ in range(2))
    qa, ka, qb, kb = empty(Hq), empty(Hkv), empty(Hq), empty(Hkv)
    us.us_norm_rope(r, q, wq, qa, k, wk, ka, off, pos, depth, max(n))
    us.us_kv_write(A, ka, v, off, pos, max(n))
    us.us_kv_append(B, r, q, wq, qb, k, wk, v, off, pos, depth, max(n), Ko=kb)
    assert us.us_get_last_device_status() == us.US_OK
    for s, t in ((A.k, B.k), (A.v, B.v), (A.scale.view(torch.int16), B.scale.view(torch.int16)), (ka.view(torch.int16), kb.view(torch.int16))):
        assert torch.equal(s, t)
    assert q is None or torch.equal(qa.view(torch.int16), qb.view(torch.int16))
    C = us.kv_cache(e, D, Hkv, page, len(ids), dev(table))
    us.us_kv_append(C, r, None, None, None, k, wk, v, off, pos, depth, max(n))          # neither queries nor dense keys
    assert torch.equal(C.k, A.k) and torch.equal(C.v, A.v)


def test_append_beside_missing_pages(us):
    x = dev(values(np.random.default_rng(6), 40, 3, 64))
    C = us.kv_cache(us.US_I8, 64, 1, 16, 4, i32([[2, 9, 1]]))
    qo = torch.zeros(40, 1, 64, dtype=torch.float16, device="cuda")
    us.us_kv_append(C, rope(us, 64, 0), x[:, :1], None, qo, x[:, 1:2], None, x[:, 2:], i32([0, 40]), i32([0]), None, 40)
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    check(qo.cpu().numpy(), x[:, :1].cpu().numpy(), None, np.arange(40), 64, 0)
    assert (C.k[2].any() and C.k[1, 0, :8].any() and not C.k[0].any() and not C.k[3].any() and not C.k[1, 0, 8:].any())
