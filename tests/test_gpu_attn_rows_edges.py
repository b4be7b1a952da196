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


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("D,H,ctx,n,at", [
    (128, 2, 0, 150, 5), (128, 2, 0, 300, 5), (64, 2, 0, 512, 200), (128, 3, 100, 300, 0), (128, 2, 100, 512, 130),
    (64, 3, 0, 300, 260), (64, 160, 0, 300, 20), (128, 100, 30, 280, 257), (64, 4, 0, 1, 0),
])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(us, what, D, H, ctx, n, at):
    """Two values of token `at` and one head, its key finite: their columns of that token and those behind it are what
    the sum is; all else is as if they were 0, on both sides of a block of 256 queries."""
    s = Setup(us, D, H, [ctx + n, 40], [n, 40], 32)
    h, cols = H - 1, [3, D - 2]
    s.V[ctx + at, h, cols] = 0
    want = s.run()
    s.check(want, heads=[0, h])
    want[at:n, h, cols] = what if np.isnan(what) else np.sign(what) * 65504
    s.V[ctx + at, h, cols] = what
    assert np.array_equal(s.run(), want, equal_nan=True)


def test_values_of_both_signs_that_are_not_finite(us):
    """Infinity less infinity, and each alone for the rows that see one of them."""
    s = Setup(us, 128, 2, [200], [200], 33)
    s.V[[50, 90], 0, 7] = 0
    want = s.run()
    s.V[50, 0, 7], s.V[90, 0, 7] = np.inf, -np.inf
    want[50:90, 0, 7], want[90:, 0, 7] = 65504, np.nan
    assert np.array_equal(s.run(), want, equal_nan=True)
