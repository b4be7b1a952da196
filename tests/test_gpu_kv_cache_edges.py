"""What the quantised cache stands for at fp16's end: rows of the largest values
read back finite."""
import numpy as np
import pytest
import torch

from oracle import kv
from tests.test_gpu_kv_cache import both, dev, offsets, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D", [64, 128])
def test_largest_values_read_back_finite(us, elem, D):
    """q times the scale of a row of 65504 is a little more than fp16 holds: what is read is 65504."""
    C, ref, rng = both(us, elem, D, 1, 16, [4], 8)
    K = rows(rng, 4, 1, D)
    K[0], K[1, 0, ::2], K[2, 0, 3], K[3, 0, 5] = 65504, -65504, np.inf, -np.inf
    V = -K[::-1].copy()
    off, at = dev(offsets([4])), dev(np.zeros(1, np.int32))
    us.us_kv_write(C, dev(K), dev(V), off, at, 4)
    out = torch.zeros(2, 4, 1, D, dtype=torch.float16, device="cuda")
    us.us_kv_read(C, off, at, 4, out[0], out[1])
    for got, x in zip(out.cpu().numpy(), (K, V)):
        c, s = kv.quantise(x, elem)
        assert np.array_equal(got, np.clip(c * s.astype(np.float64)[..., None], -65504, 65504).astype(np.float16))
