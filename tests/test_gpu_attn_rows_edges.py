"""Causal attention over expanded rows at its edges: references that move with every tile,
and what stands between the threads that share a row."""
import numpy as np
import pytest

from tests.test_gpu_attn_rows import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("H,kv,n", [(1, [300], [300]), (24, [3000, 700], [256, 300]), (40, [1500], [512])])
def test_outputs_that_are_rescaled_with_every_tile(us, D, H, kv, n):
    """A tile's scores lie 11 to 13 (2^16 to 2^19 in weights) above the last one's, so that all columns of the
    outputs, which two threads hold, are scaled down before each product that adds to them."""
    s = Setup(us, D, H, kv, n, 31)
    for L, at in zip(kv, np.cumsum([0] + kv)):
        s.R[at:at + L] = 0
        s.R[at:at + L, 0] = 12.0 / (20 * s.scale) * (np.arange(L) // 128)
    s.Q[..., D] = 20.0
    ws = us.workspace_attn_rows(D, 64, D, H, len(n), max(n))
    got = s.run(ws=ws)
    s.check(got, heads=[0, H // 2, H - 1])
    for _ in range(5):
        assert np.array_equal(got, s.run(ws=ws))
