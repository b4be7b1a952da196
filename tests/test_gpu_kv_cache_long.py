"""Long writes and reads of the quantised cache: every (token, head) row of a
thread's several, CTAs of many tokens, ragged ends.  Stored bytes and values
read back are exact."""
import numpy as np
import pytest
import torch

from oracle import kv
from tests.test_gpu_kv_cache import both, dev, offsets, rows, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,counts,pos", [
    (128, 32, [900, 611], [0, 77]), (64, 32, [611, 0, 450], [3, 0, 16]), (128, 5, [2000, 1, 1333], [5, 0, 100]),
    (64, 5, [2700, 2601, 64], [0, 63, 1]), (128, 1, [9800, 9500], [31, 0]), (64, 1, [20000, 18999], [0, 1]),
    (128, 40, [3, 0, 17], [0, 1, 15]), (64, 67, [2, 5], [62, 0]),
])
def test_write_and_read_back(us, elem, D, Hkv, counts, pos):
    page = 64
    C, ref, rng = both(us, elem, D, Hkv, page, [p + n for p, n in zip(pos, counts)], 7)
    T = sum(counts)
    K, V = rows(rng, T, Hkv, D), rows(rng, T, Hkv, D)
    p = np.concatenate([np.arange(a, a + n) for a, n in zip(pos, counts)])
    b = np.repeat(np.arange(len(counts)), counts)
    pages, slots = ref.table[b, p // page], p % page
    want = []
    for i, (pool, x) in enumerate(((ref.k, K), (ref.v, V))):
        c, s = kv.quantise(x, elem)
        pool[pages, :, slots], ref.scale[pages, :, slots, i] = kv.pack(c, elem), s
        want.append((c * s.astype(np.float64)[..., None]).astype(np.float16))
    off, at = dev(offsets(counts)), dev(np.array(pos, np.int32))
    us.us_kv_write(C, dev(K), dev(V), off, at, max(counts))
    same(C, ref)
    out = torch.zeros(2, T, Hkv, D, dtype=torch.float16, device="cuda")
    us.us_kv_read(C, off, at, max(counts), out[0], out[1])
    got = out.cpu().numpy()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert us.us_get_last_device_status() == us.US_OK
