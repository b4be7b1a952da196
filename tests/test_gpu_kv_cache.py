"""The quantised K/V cache on the GPU against the plain reference: stored bytes,
values read back and committed paths are exact."""
import numpy as np
import pytest
import torch

from oracle import kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def both(us, elem, D, Hkv, page, lens, seed, spare=2):
    """An empty cache here and in the reference, over the same shuffled pages."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 1) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    ref = kv.Cache(elem, D, Hkv, page, len(ids), table)
    return us.kv_cache(elem, D, Hkv, page, len(ids), dev(table)), ref, rng


def offsets(counts):
    return np.concatenate(([0], np.cumsum(counts))).astype(np.int32)


def rows(rng, T, H, D):
    x = rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1)))
    x[..., 0] *= 8
    return x.astype(np.float16)


def same(C, ref):
    torch.cuda.synchronize()
    assert np.array_equal(C.k.cpu().numpy(), ref.k) and np.array_equal(C.v.cpu().numpy(), ref.v)
    assert np.array_equal(C.scale.cpu().numpy().view(np.uint16), ref.scale.view(np.uint16))


def write(us, C, ref, K, V, counts, pos, pad=0):
    """Write through the library (rows `pad` elements apart) and in the reference."""
    T, H, D = K.shape
    buf = torch.zeros(T, 2 * H * D + pad, dtype=torch.float16, device="cuda")
    buf[:, :H * D], buf[:, H * D:2 * H * D] = dev(K).reshape(T, -1), dev(V).reshape(T, -1)
    kd, vd = (buf[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (0, 1))
    us.us_kv_write(C, kd, vd, dev(offsets(counts)), dev(np.array(pos, np.int32)), max(counts))
    t = 0
    for b, n in enumerate(counts):
        for i in range(n):
            ref.write(b, pos[b] + i, K[t], V[t])
            t += 1


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,page,counts,pos", [
    (128, 8, 64, [1], [0]),
    (128, 1, 16, [1, 1, 1], [15, 16, 999]),
    (64, 3, 16, [0, 37, 5], [4, 11, 0]),
    (128, 5, 32, [130, 0, 1, 61], [0, 7, 31, 33]),
    (64, 32, 128, [17, 33], [127, 300]),
])
def test_write_and_read_back(us, elem, D, Hkv, page, counts, pos):
    C, ref, rng = both(us, elem, D, Hkv, page, [p + n for p, n in zip(pos, counts)], 1)
    T = sum(counts)
    K, V = rows(rng, T, Hkv, D), rows(rng, T, Hkv, D)
    write(us, C, ref, K, V, counts, pos, pad=24)
    same(C, ref)
    out = torch.zeros(2, T, Hkv, D, dtype=torch.float16, device="cuda")
    us.us_kv_read(C, dev(offsets(counts)), dev(np.array(pos, np.int32)), max(counts), out[0], out[1])
    want = [ref.read(b, pos[b] + i) for b, n in enumerate(counts) for i in range(n)]
    got = out.cpu().numpy()
    assert np.array_equal(got[0], np.array([w[0] for w in want]).astype(np.float16))
    assert np.array_equal(got[1], np.array([w[1] for w in want]).astype(np.float16))
    assert us.us_get_last_device_status() == us.US_OK


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
def test_rows_of_special_values(us, elem):
    """Zeros, the largest and smallest magnitudes, infinities, NaN and exact ties."""
    D = 64
    C, ref, rng = both(us, elem, D, 1, 16, [9], 2)
    K = np.zeros((9, 1, D), np.float16)
    q = kv.QMAX[elem]
    K[1] = np.float16(65504)
    K[2, 0, :4] = [np.inf, -np.inf, np.nan, 1]
    K[3, 0, :3] = [5.96e-8, -5.96e-8, 0]                       # one subnormal step
    K[4, 0, :6] = np.array([q, 0.5, 1.5, 2.5, -0.5, -3.5])     # scale 1: ties go to even
    K[5, 0, :] = -0.0
    K[6, 0, :] = np.nan
    K[7, 0, :] = (np.arange(D) - 32) * 3e-7                    # scale rounds among subnormals
    K[8, 0, :] = rng.standard_normal(D) * 1e-3
    write(us, C, ref, K, K[::-1].copy(), [9], [0])
    same(C, ref)
    assert np.isfinite(C.scale.float().cpu().numpy()).all()


def test_overwriting_leaves_neighbours(us):
    """A second write to some positions changes those entries alone (int4 shares no byte between entries)."""
    C, ref, rng = both(us, kv.I4, 128, 2, 16, [40, 40], 3)
    write(us, C, ref, rows(rng, 80, 2, 128), rows(rng, 80, 2, 128), [40, 40], [0, 0])
    write(us, C, ref, rows(rng, 3, 2, 128), rows(rng, 3, 2, 128), [1, 2], [15, 31])
    same(C, ref)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,page", [(128, 8, 64), (64, 3, 16)])
def test_commit(us, elem, D, Hkv, page):
    """Paths that overlap themselves, cross pages, stay in place, reverse, or are empty."""
    paths = [[0, 2, 3, 7], [], [0], [5, 6, 7, 8, 9, 10], list(range(20)), [3, 2, 1, 0], list(range(1, 64)) + [0]]
    pos = [14, 3, 0, 15, 30, 61, 5]
    lens = [p + 64 for p in pos]
    C, ref, rng = both(us, elem, D, Hkv, page, lens, 4)
    counts = [64] * len(pos)
    write(us, C, ref, rows(rng, sum(counts), Hkv, D), rows(rng, sum(counts), Hkv, D), counts, pos)
    off = offsets([len(p) for p in paths])
    us.us_kv_commit(C, dev(off), dev(np.array(sum(paths, []), np.int32)), dev(np.array(pos, np.int32)), 64)
    for b, path in enumerate(paths):
        ref.commit(b, pos[b], path)
    same(C, ref)
    assert us.us_get_last_device_status() == us.US_OK


def test_bad_pages_and_offsets_are_recorded_and_skipped(us):
    C, ref, rng = both(us, kv.I8, 64, 2, 16, [64, 64], 5)
    K, V = rows(rng, 128, 2, 64), rows(rng, 128, 2, 64)
    write(us, C, ref, K, V, [64, 64], [0, 0])
    bad = us.KVCache(C.elem, C.D, C.k, C.v, C.scale, C.page_table.clone())
    bad.page_table[1, 2] = C.k.shape[0]                        # one past the last page
    one = dev(np.array([0, 0], np.int32))
    out = torch.full((2, 128, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    us.us_kv_read(bad, dev(offsets([64, 64])), one, 64, out[0], out[1])
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    got = out.cpu().numpy()
    assert (got[:, 96:112] == 7).all()                         # that page's positions are left alone
    assert np.array_equal(got[0, 64:96], np.array([ref.read(1, p)[0] for p in range(32)]).astype(np.float16))
    kd, vd = dev(K), dev(V)
    for off, pos in (([0, 64, 63], [0, 0]), ([0, 64, 129], [0, 0]), ([-1, 64, 128], [0, 0]),
                     ([0, 0, 128], [0, 0]), ([0, 1, 2], [80, -5]), ([0, 1, 2], [2**31 - 1, 0])):
        us.us_kv_write(C, kd, vd, dev(np.array(off, np.int32)), dev(np.array(pos, np.int32)), 64)
        assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
    acc = dev(np.array([0, -1, 1000], np.int32))
    us.us_kv_commit(C, dev(np.array([0, 3, 3], np.int32)), acc, one, 3)
    assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG


def test_captured_graph_follows_positions(us):
    C, ref, rng = both(us, kv.I4, 128, 2, 16, [50], 6)
    K, V = dev(rows(rng, 1, 2, 128)), dev(rows(rng, 1, 2, 128))
    off, pos = dev(offsets([1])), dev(np.array([0], np.int32))
    out = torch.zeros(2, 1, 2, 128, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        us.us_kv_write(C, K, V, off, pos, 1)
        us.us_kv_read(C, off, pos, 1, out[0], out[1])
    for p in (0, 17, 49):
        k, v = rows(rng, 1, 2, 128), rows(rng, 1, 2, 128)
        K.copy_(dev(k)), V.copy_(dev(v))
        pos.fill_(p)
        graph.replay()
        ref.write(0, p, k[0], v[0])
        want = ref.read(0, p)
        assert np.array_equal(out.cpu().numpy()[:, 0], np.array(want).astype(np.float16))
    same(C, ref)
