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


@pytest.mark.parametrize("Dc,Hq,ctx", [(512, 16, 0), (256, 64, 0), (512, 4, 700)])
@pytest.mark.parametrize("size", [40, 120, 250, 1000, 2000, 4000, 20000, 60000])
def test_large_scores(us, Dc, Hq, ctx, size):
    """Entries of one direction and steadily different lengths, which queries of both signs rank: each row's output is the
    first or the last entry.  Scores are a tenth of themselves apart at the ends, and from 2^9 to beyond 2^30."""
    s = Setup(us, Dc, Hq, 16, [ctx], [1], 43)
    along = np.sign(s.rng.standard_normal(s.W))
    for order in (1, -1):
        length = np.full(ctx + 1, 1.0)
        length[0] = 0.8 if order > 0 else 1.0
        length[1:] = np.linspace(0.85, 0.95, ctx) if ctx else 0
        length[ctx] = 1.0 if order > 0 or not ctx else 0.8
        for p in range(ctx + 1):
            put(s, 0, p, (size * length[p] * along).astype(np.float16))
        s.load()
        s.Q[:] = (size * along * np.where(np.arange(Hq) % 2, -1, 1)[:, None]).astype(np.float16)
        got, rows = s.run(None)[0], s.rows(0).astype(np.float64)[:, :Dc]
        # the next best score lies 0.05 size^2 W scale away: a weight of e^-60 and less from size 40 on
        best = np.abs(rows[:, 0])
        for h in range(Hq):
            want = rows[best.argmax() if h % 2 == 0 else best.argmin()]
            assert (np.abs(got[h] - want) <= 2.0 ** -10 * np.abs(want)).all()


@pytest.mark.parametrize("Hq", [2, 64])
@pytest.mark.parametrize("base", [512, 1024, 2048, 4096])
def test_large_scores_close_to_one_another(us, Hq, base):
    """Scores of 2^20 to 2^23 (base 1024) that rise by a little from tile to tile: outputs are weighted means."""
    for step in (3.3, 3.4, 3.5, 3.6, 7.0, 11.0):
        s = Setup(us, 256, Hq, 64, [191], [1], 44)
        for p in range(192):
            put(s, 0, p, 0, slice(256, 320))
            put(s, 0, p, [base, step * (p // 64)], slice(256, 258))
        s.load()
        s.Q[:] = 0
        s.Q[..., 256], s.Q[..., 257], s.scale = 1024, 1, 1.0
        got, most = s.run(None), np.abs(s.rows(0)[:, :256].astype(np.float64)).max()
        assert (np.abs(got) <= most * (1 + 2.0 ** -9)).all()
