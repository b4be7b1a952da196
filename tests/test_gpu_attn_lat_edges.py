"""Attention over latent rows at its edges: what rows do not see, and what they see that is not finite."""
import numpy as np
import pytest

from tests.test_gpu_attn_lat import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def put(s, b, p, what, cols=slice(None)):
    s.pool[s.table[b, p // s.page], p % s.page, cols] = what


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("Dc,Hq", [(512, 16), (256, 64), (512, 1)])
def test_single_tokens_that_do_not_see_themselves(us, what, Dc, Hq):
    """A batch of fixed size, some of whose requests are padding: masks of 0 and entries that were never written."""
    ctx = [0, 70, 0, 63, 64, 300]
    s = Setup(us, Dc, Hq, 16, ctx, [1] * len(ctx), 41)
    words = np.array([0, 0, 1, 0, 0, 1], np.int64)
    grids = [[[int(w)]] for w in words]
    for b in np.flatnonzero(words == 0):
        put(s, b, ctx[b], what)
    s.load()
    got = s.run(words)
    s.check(got, grids)
    assert (got[0] == 0).all() and (got[1] != 0).any()
