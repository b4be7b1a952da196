"""The cache of latent rows on the GPU: writing against the plain reference in 64 bits
(tolerance as for norm and rotation of heads), reading back and committing exactly."""
import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_gpu_kv_cache import dev, offsets
from tests.test_gpu_rope import EPS, check, i32, rope, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def make(us, Dc, page, lens, seed, spare=2):
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 1) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    for b, m in enumerate(need):
        table[b, :m] = ids[sum(need[:b]):sum(need[:b + 1])]
    C = us.lat_cache(Dc, 64, page, len(ids), dev(table))
    C.rows.fill_(5.0)
    return C, table, rng


def entry(C, table, b, p):
    page = C.page_size
    return C.rows[int(table[b, p // page]), p % page]


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("Dc,page,n,ctx,normed,R", [
    (512, 16, [1] * 5, [0, 15, 16, 17, 100], True, 64),
    (256, 64, [70, 0, 3], [0, 9, 63], True, 64),
    (512, 64, [129], [1000], False, 64),
    (512, 32, [8, 9], [130000, 2], True, 64),
    (256, 16, [20], [5], True, 0),
])
def test_write_and_read(us, style, Dc, page, n, ctx, normed, R):
    C, table, rng = make(us, Dc, page, [c + m for c, m in zip(ctx, n)], Dc + page)
    T, W = sum(n), Dc + 64
    x = values(rng, T, 1, W)[:, 0]
    w = (1 + 0.3 * rng.standard_normal(Dc)).astype(np.float16) if normed else None
    wide = torch.zeros(T, W + 24, dtype=torch.float16, device="cuda")
    wide[:, :W] = dev(x)
    off, pos, r = dev(offsets(n)), i32(ctx), rope(us, R, style)
    depth = rng.integers(0, 30, T)
    for dd in (None, depth):
        C.rows.fill_(5.0)
        us.us_lat_write(C, r, wide[:, :W], None if w is None else dev(w), off, pos, None if dd is None else i32(dd), max(n) + 3)
        out = torch.full((T + 1, W + 8), 7.0, dtype=torch.float16, device="cuda")
        us.us_lat_read(C, off, pos, max(n), out[:T, :W])
        assert us.us_get_last_device_status() == us.US_OK
        p = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, n)])
        at = p if dd is None else np.concatenate([np.full(m, c) for c, m in zip(ctx, n)]) + dd
        got = out[:T, :W].cpu().numpy()
        check(got[:, None, :Dc], x[:, None, :Dc], w, p, 0, 0)
        check(got[:, None, Dc:], x[:, None, Dc:], None, at, R, style)
        assert (out[T] == 7).all() and (out[:T, W:] == 7).all()
        t = 0
        for b, m in enumerate(n):
            for i in range(m):
                assert torch.equal(entry(C, table, b, ctx[b] + i), out[t, :W])
                t += 1
        assert int((C.rows != 5).any(-1).sum()) == T                # nothing else was written


def test_what_is_stored_is_finite(us):
    C, table, rng = make(us, 256, 16, [6], 1)
    x = values(rng, 6, 1, 320)[:, 0]
    x[1, 3], x[2, 7], x[3, 260], x[4, 300] = np.inf, np.nan, np.nan, -np.inf
    x[5, :256] = 65504
    w = np.full(256, 3.0, np.float16)
    us.us_lat_write(C, rope(us, 64, 1), dev(x), dev(w), i32([0, 6]), i32([0]), None, 6)
    assert us.us_get_last_device_status() == us.US_OK
    out = torch.zeros(6, 320, dtype=torch.float16, device="cuda")
    us.us_lat_read(C, i32([0, 6]), i32([0]), 6, out)
    got = out.cpu().numpy()
    assert np.isfinite(got).all()
    check(got[5:, None, :256], x[5:, None, :256], w, [5], 0, 0)
    big = np.full((1, 320), 60000.0, np.float16)
    us.us_lat_write(C, rope(us, 64, 0), dev(big), None, i32([0, 1]), i32([3]), None, 1)    # 60000 (cos + sin) is beyond fp16
    us.us_lat_read(C, i32([0, 1]), i32([3]), 1, out[:1])
    got = out[:1].cpu().numpy()
    assert np.isfinite(got).all() and np.abs(got[0, 256:]).max() == 65504


def test_commit(us):
    for Dc, page in ((512, 16), (256, 64)):
        ctx, n = [30, 0, 15, 100], [20, 64, 1, 9]
        C, table, rng = make(us, Dc, page, [c + m for c, m in zip(ctx, n)], 7)
        C.rows.copy_(dev(rng.standard_normal(C.rows.shape).astype(np.float16)))
        before = C.rows.clone()
        acc = [sorted(rng.choice(m, min(m, 7), replace=False).tolist()) for m in n[:2]] + [[0], [8, 8, 0, 3]]
        us.us_lat_commit(C, dev(offsets([len(a) for a in acc])), i32(sum(acc, [])), i32(ctx), 7)
        assert us.us_get_last_device_status() == us.US_OK
        want = before.clone()
        for b, a in enumerate(acc):
            for i, d in enumerate(a):
                p, s = ctx[b] + i, ctx[b] + d
                want[int(table[b, p // page]), p % page] = before[int(table[b, s // page]), s % page]
        assert torch.equal(C.rows, want)


def test_bad_pages_and_positions(us):
    C, table, rng = make(us, 256, 16, [64], 8)
    C.page_table[0, 1] = 99
    x = dev(values(rng, 40, 1, 320)[:, 0])
    us.us_lat_write(C, rope(us, 64, 0), x, None, i32([0, 40]), i32([0]), None, 40)
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    out = torch.full((40, 320), 7.0, dtype=torch.float16, device="cuda")
    us.us_lat_read(C, i32([0, 40]), i32([0]), 40, out)
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    assert torch.equal(out[:16, :256], x[:16, :256]) and torch.equal(out[32:, :256], x[32:, :256]) and (out[16:32] == 7).all()
    before = C.rows.clone()
    for pos in (-3, 16 * 5, 2 ** 31 - 1):
        us.us_lat_write(C, rope(us, 64, 0), x[:1], None, i32([0, 1]), i32([pos]), None, 1)
        assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
    us.us_lat_commit(C, i32([0, 2]), i32([-1, 20]), i32([0]), 2)
    assert us.us_get_last_device_status() != us.US_OK
    assert torch.equal(C.rows, before)


def test_entries_beyond_32_bit_offsets(us):
    """A pool of 4.6 GB: the last page's rows lie beyond 2^31 values."""
    pages = 4_000_000_000 // (576 * 64) // 2 * 2 + 9000
    table = i32([[pages - 1, 0, pages - 2]])
    C = us.LatCache(512, 64, torch.empty(pages, 64, 576, dtype=torch.float16, device="cuda"), table)
    assert C.rows.numel() > 2 ** 32
    C.rows[pages - 1].zero_(), C.rows[pages - 2].zero_(), C.rows[0].zero_()
    rng = np.random.default_rng(9)
    x = dev(values(rng, 150, 1, 576)[:, 0])
    us.us_lat_write(C, rope(us, 0, 0), x, None, i32([0, 150]), i32([0]), None, 150)
    out = torch.zeros_like(x)
    us.us_lat_read(C, i32([0, 150]), i32([0]), 150, out)
    assert us.us_get_last_device_status() == us.US_OK
    assert torch.equal(out, x) and torch.equal(C.rows[pages - 1], x[:64]) and torch.equal(C.rows[0], x[64:128])
    # and the attention reads them
    q = dev((0.1 * rng.standard_normal((1, 16, 576))).astype(np.float16))
    o = torch.zeros(1, 16, 512, dtype=torch.float16, device="cuda")
    us.us_attn_lat(C, q, i32([0, 1]), i32([149]), None, 1, 0.07, o, us.workspace_attn_lat(C, 16, 1))
    assert us.us_get_last_device_status() == us.US_OK
    s = torch.softmax(q[0].double() @ x.double().T * 0.07, -1)
    assert (o[0].double() - s @ x[:, :512].double()).abs().max() <= 2e-3 * x.abs().max().item()


def test_a_limit_far_beyond_the_rows(us):
    """max_n is a promise, not a size: 2^30 - 1 of it gives what the rows' own number gives."""
    n, most = 37, (1 << 30) - 1
    C, table, rng = make(us, 256, 16, [n + 5], 77)
    x, w = dev(values(rng, n, 1, 320)[:, 0]), dev((1 + 0.3 * rng.standard_normal(256)).astype(np.float16))
    off, pos, r = dev(offsets([n])), i32([5]), rope(us, 64, 0)
    q = dev(values(rng, n, 4, 64))
    P = us.kv_pool(16, 8, 1, 4)
    us.us_kv_reserve(P, i32([n + 5]))
    C.rows.fill_(0)                                                # (what the call does not write is seen, too)
    got = {}
    for m in (n, most):
        rows, o = torch.zeros(n, 320, dtype=torch.float16, device="cuda"), torch.zeros(n, 4, 256, dtype=torch.float16, device="cuda")
        qo, slots = torch.zeros_like(q), torch.zeros(n, dtype=torch.int64, device="cuda")
        us.us_lat_write(C, r, x, w, off, pos, None, m)
        us.us_lat_read(C, off, pos, m, rows)
        us.us_norm_rope(r, q, None, qo, None, None, None, off, pos, None, m)
        us.us_kv_slots(P, off, pos, m, slots)
        m4 = min(m, most // 4)
        us.us_attn_lat(C, rows.unflatten(1, (1, 320)).expand(n, 4, 320).contiguous(), off, pos, None, m4, 0.05, o, us.workspace_attn_lat(C, 4, m4))
        assert us.us_get_last_device_status() == us.US_OK
        got[m] = [t.cpu() for t in (rows, qo, slots, o)]
    assert got[n][0].abs().max() > 0 and all(torch.equal(a, b) for a, b in zip(got[n], got[most]))
