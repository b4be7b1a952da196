"""The cache of latent rows at its edges."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import dev
from tests.test_gpu_lat import make
from tests.test_gpu_rope import i32, rope, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("what,stored", [(np.inf, 65504), (-np.inf, -65504), (np.nan, 0)])
@pytest.mark.parametrize("Dc", [256, 512])
def test_without_rotation_a_value_that_is_not_finite_stands_alone(us, what, stored, Dc):
    """Neither norm nor rotation: each value is stored as it is, made finite by itself."""
    C, table, rng = make(us, Dc, 16, [3], 2)
    x = values(rng, 3, 1, Dc + 64)[:, 0]
    at = [(0, 5), (0, Dc), (1, Dc + 1), (1, Dc + 40), (2, Dc + 63)]
    want = x.copy()
    for t, c in at:
        x[t, c], want[t, c] = what, stored
    for style in (0, 1):
        us.us_lat_write(C, rope(us, 0, style), dev(x), None, i32([0, 3]), i32([0]), None, 3)
        assert us.us_get_last_device_status() == us.US_OK
        out = torch.zeros(3, Dc + 64, dtype=torch.float16, device="cuda")
        us.us_lat_read(C, i32([0, 3]), i32([0]), 3, out)
        assert np.array_equal(out.cpu().numpy(), want)
