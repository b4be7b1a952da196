"""Page tables and slots worked out on the GPU against the plain pool: all whole numbers, all equal."""
import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_gpu_kv_cache import dev, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def i32(v):
    return dev(np.array(v, np.int32))


def same(P, ref):
    torch.cuda.synchronize()
    assert np.array_equal(P.page_table.cpu().numpy(), ref.table())
    assert P.held.cpu().tolist() == [len(x) for x in ref.held]
    n = int(P.free_count.cpu())
    assert P.free_pages.cpu().tolist()[:n] == ref.free


@pytest.mark.parametrize("page,num_pages,B,max_pages,top", [
    (16, 40, 1, 40, 700), (16, 500, 7, 64, 1000), (64, 3000, 130, 40, 2500), (1024, 50, 33, 3, 3000), (16, 60000, 1024, 100, 1600)])
def test_lengths_that_come_and_go(us, page, num_pages, B, max_pages, top):
    rng = np.random.default_rng(B)
    P, ref = us.kv_pool(page, num_pages, B, max_pages), lat.Pool(page, num_pages, B, max_pages)
    same(P, ref)
    for step in range(6):
        n = rng.integers(0, top + 1, B) * (rng.random(B) < 0.8)
        n = np.minimum(n, max_pages * page)
        while sum(-(-n // page)) > num_pages:
            n //= 2
        us.us_kv_reserve(P, i32(n))
        assert ref.reserve(n.tolist())
        same(P, ref)
    assert us.us_get_last_device_status() == us.US_OK


def test_exact_page_ends(us):
    P, ref = us.kv_pool(16, 30, 5, 8), lat.Pool(16, 30, 5, 8)
    for n in ([0, 1, 15, 16, 17], [16, 16, 16, 16, 16], [17, 32, 33, 128, 0], [0] * 5, [128, 128, 128, 96, 0], [128, 128, 128, 96, 0]):
        us.us_kv_reserve(P, i32(n))
        assert ref.reserve(n)
        same(P, ref)
    assert us.us_get_last_device_status() == us.US_OK


def test_too_few_pages(us):
    """In order: from the first request that does not fit, those that want more get none."""
    P, ref = us.kv_pool(16, 10, 4, 8), lat.Pool(16, 10, 4, 8)
    for n, fits in (([32, 32, 16, 0], True), ([16, 128, 16, 16], False), ([48, 64, 0, 16], True), ([48, 64, 16, 128], False), ([0, 0, 0, 0], True)):
        us.us_kv_reserve(P, i32(n))
        assert ref.reserve(n) == fits
        same(P, ref)
        assert us.us_get_last_device_status() == (us.US_OK if fits else us.US_ERR_WORKSPACE)


def test_bad_lengths_leave_the_request(us):
    P, ref = us.kv_pool(16, 20, 3, 4), lat.Pool(16, 20, 3, 4)
    us.us_kv_reserve(P, i32([20, 20, 20]))
    ref.reserve([20, 20, 20])
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        us.us_kv_reserve(P, i32([40, bad, 1]))
        ref.reserve([40, 20, 1])
        same(P, ref)
        assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value", [("free_count", -1), ("free_count", 21), ("held", -1), ("held", 5), ("free_count", 20)])
def test_corrupt_pools_are_left_alone(us, field, value):
    """(A full stack while pages are held: more would be given back than there is room for.)"""
    P = us.kv_pool(16, 20, 3, 4)
    us.us_kv_reserve(P, i32([20, 40, 0]))
    getattr(P, field)[-1 if field == "held" else 0] = value
    before = [t.clone() for t in (P.page_table, P.held, P.free_pages, P.free_count)]
    us.us_kv_reserve(P, i32([0, 16, 20]))
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    for t, u in zip((P.page_table, P.held, P.free_pages, P.free_count), before):
        assert torch.equal(t, u)


@pytest.mark.parametrize("page,n", [(16, [3, 0, 40, 1]), (64, [300, 1, 0, 513])])
def test_slots(us, page, n):
    ctx = [5, 70, 0, 16]
    P, ref = us.kv_pool(page, 200, 4, 80), lat.Pool(page, 200, 4, 80)
    need = [c + k for c, k in zip(ctx, n)]
    us.us_kv_reserve(P, i32([9, 999, 0, 300]))
    us.us_kv_reserve(P, i32(need))
    ref.reserve([9, 999, 0, 300])
    ref.reserve(need)
    got = torch.full((sum(n) + 3,), -7, dtype=torch.int64, device="cuda")
    us.us_kv_slots(P, dev(offsets(n)), i32(ctx), max(n), got)
    want = [ref.slot(b, ctx[b] + i) for b in range(4) for i in range(n[b])]
    assert got.cpu().tolist() == want + [-7] * 3                  # rows behind the last token stay
    assert us.us_get_last_device_status() == us.US_OK


def test_slots_where_there_is_no_page(us):
    P = us.kv_pool(16, 20, 3, 4)
    us.us_kv_reserve(P, i32([16, 64, 10]))
    got = torch.full((12,), -7, dtype=torch.int64, device="cuda")
    us.us_kv_slots(P, i32([0, 4, 8, 12]), i32([14, 62, -2]), 4, got)
    t = P.page_table.cpu()
    assert got.cpu().tolist() == [int(t[0, 0]) * 16 + 14, int(t[0, 0]) * 16 + 15, -1, -1, int(t[1, 3]) * 16 + 14, int(t[1, 3]) * 16 + 15, -1, -1,
                                  -1, -1, int(t[2, 0]) * 16, int(t[2, 0]) * 16 + 1]
    assert us.us_get_last_device_status() in (us.US_ERR_CORRUPT, us.US_ERR_INVALID_ARG)
    us.us_kv_slots(P, i32([0, 4, 3, 12]), i32([0, 0, 0]), 4, got)   # offsets that do not ascend: the others are done
    assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
    assert got.cpu().tolist()[:4] == [int(t[0, 0]) * 16 + i for i in range(4)]


def test_captured_and_replayed(us):
    """A graph follows the lengths' values; the table serves a cache."""
    P, ref = us.kv_pool(16, 64, 3, 16), lat.Pool(16, 64, 3, 16)
    n, pos, off = i32([1, 20, 33]), i32([0, 19, 32]), i32([0, 1, 2, 3])
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        us.us_kv_reserve(P, n)
        us.us_kv_slots(P, off, pos, 1, slots)
    torch.cuda.current_stream().wait_stream(side)
    ref.reserve([1, 20, 33])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        us.us_kv_reserve(P, n)
        us.us_kv_slots(P, off, pos, 1, slots)
        n += 7
        pos += 7
    lens = np.array([1, 20, 33])
    for _ in range(20):
        g.replay()
        ref.reserve(lens.tolist())
        same(P, ref)
        assert slots.cpu().tolist() == [ref.slot(b, lens[b] - 1) for b in range(3)]
        lens = lens + 7
    assert us.us_get_last_device_status() == us.US_OK


def test_threads_that_have_not_used_the_device(us):
    """Calls from new threads, several at once, each on a stream and a pool of its own."""
    import threading
    pools = [us.kv_pool(16, 200, 4, 50) for _ in range(8)]
    refs = [lat.Pool(16, 200, 4, 50) for _ in range(8)]
    lens = [[10 * i, 700, 0, 33 + i] for i in range(8)]
    at, streams, errors = [i32(n) for n in lens], [torch.cuda.Stream() for _ in range(8)], []
    torch.cuda.synchronize()

    def work(i):
        try:
            us.us_kv_reserve(pools[i], at[i], streams[i])
        except Exception as e:                                     # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and us.us_get_last_device_status() == us.US_OK
    for P, ref, n in zip(pools, refs, lens):
        ref.reserve(n)
        same(P, ref)
