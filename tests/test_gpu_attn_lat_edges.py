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


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("Dc,Hq,ctx,n,at,col", [
    (512, 4, 20, 6, 22, 100), (256, 64, 90, 9, 91, 3), (512, 16, 0, 64, 30, 511), (512, 4, 20, 6, 5, 100), (256, 8, 300, 3, 10, 260),
    (512, 2, 30, 5, 32, 575),
])
def test_entries_that_are_not_finite_make_nan_of_the_rows_that_see_them(us, what, Dc, Hq, ctx, n, at, col):
    """One value of one entry, of the context or of the call's tokens, latent or of the key, and queries of both signs there."""
    for tree in (False, True):
        s = Setup(us, Dc, Hq, 16, [ctx], [n], 42)
        words, grids = s.tree() if tree else s.chain()
        s.Q[..., col] = np.where(np.arange(Hq) % 2, 1, -1)
        want = s.run(words)
        s.check(want, grids)
        put(s, 0, at, what, col)
        s.load()
        sees = np.ones(n, bool) if at < ctx else np.array(grids[0], bool)[:, at - ctx]
        got = s.run(words)
        assert np.isnan(got[sees]).all() and np.array_equal(got[~sees], want[~sees]) and sees.any()
