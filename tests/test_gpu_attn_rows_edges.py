"""Causal attention over expanded rows at its edges: references that move with every tile,
and what stands between the threads that share a row."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attn_rows import Setup
from tests.test_gpu_kv_cache import dev
from tests.test_gpu_rope import i32

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


@pytest.mark.parametrize("D,H,ctx,n", [(128, 2, 0, 1), (64, 2, 0, 1), (128, 3, 400, 1), (64, 40, 700, 3)])
@pytest.mark.parametrize("size", [60, 250, 1000, 2000, 4000, 7000, 20000, 60000])
def test_large_scores(us, D, H, ctx, n, size):
    """Keys of one direction and steadily different lengths, which queries of both signs rank: each row's output is the value
    of the first position or of its own.  Scores from 2^10 to beyond 2^30."""
    s = Setup(us, D, H, [ctx + n], [n], 34)
    L, along = ctx + n, np.sign(s.rng.standard_normal(D + 64))
    for order in (1, -1):
        length = np.linspace(0.85, 0.9, L)
        length[0], length[ctx:] = (0.8, 0.95 + 0.05 * np.arange(n) / 3) if order > 0 else (1.0, 0.8 - 0.05 * np.arange(n) / 3)
        key = (size * length[:, None] * along).astype(np.float16)
        s.K[:], s.R[:] = key[:, None, :D], key[:, D:]
        s.Q[:] = (size * along * np.where(np.arange(H) % 2, -1, 1)[:, None]).astype(np.float16)
        got = s.run()
        # the next best score lies 0.016 size^2 (D + 64) scale away: a weight of e^-600 and less from size 60 on
        for i in range(n):
            for h in range(H):
                want = s.V[ctx + i if (h % 2 == 0) == (order > 0) else 0, h].astype(np.float64)
                assert (np.abs(got[i, h] - want) <= 2.0 ** -10 * np.abs(want) + 2.0 ** -24).all()


@pytest.mark.parametrize("H", [1, 64])
@pytest.mark.parametrize("base", [512, 1024, 2048, 4096])
def test_large_scores_close_to_one_another(us, H, base):
    """Scores of 2^20 to 2^23 (base 1024) that rise by a little from tile to tile: outputs are weighted means."""
    for step in (3.3, 3.4, 3.5, 3.6, 7.0, 11.0):
        s = Setup(us, 64, H, [384], [200], 35)
        s.R[:] = 0
        s.R[:, 0], s.R[:, 1] = base, step * (np.arange(384) // 128)
        s.Q[:] = 0
        s.Q[..., 64], s.Q[..., 65], s.scale = 1024, 1, 1.0
        got, most = s.run(), np.abs(s.V.astype(np.float64)).max()
        assert (np.abs(got) <= most * (1 + 2.0 ** -9)).all()


@pytest.mark.parametrize("D,H,kv,n", [(128, 1, [4000], [3]), (64, 2, [3000, 500], [20, 1])])
def test_a_limit_far_beyond_the_rows(us, D, H, kv, n):
    """max_n is a promise: beyond the rows of the call it has no part in how states are joined."""
    s = Setup(us, D, H, kv, n, 36)
    got = s.run(max_n=sum(n))
    s.check(got)
    for max_n in (sum(n) + 1, 5000, 1 << 28):
        assert np.array_equal(got, s.run(max_n=max_n))


def test_key_offsets_of_requests_without_queries_are_checked(us):
    """Offsets that do not ascend or leave 0..S are recorded whichever request they are of; the others are served."""
    s = Setup(us, 64, 2, [40, 30, 60], [20, 0, 30], 37)
    good = s.run()
    o = torch.zeros(50, 2, 64, dtype=torch.float16, device="cuda")
    ws = us.workspace_attn_rows(64, 64, 64, 2, 3, 30)
    for off, kv_off, code, kept in (
            ([0, 20, 20, 50], [0, 40, 70, 130], us.US_OK, [(0, 50)]),
            ([0, 20, 20, 50], [0, 40, 40, 130], us.US_OK, [(0, 20)]),               # no key rows either: the last one has 90
            ([0, 20, 20, 50], [0, 80, 70, 130], us.US_ERR_INVALID_ARG, [(20, 50)]),  # (the first one has 80)
            ([0, 20, 50, 50], [0, 40, 100, 131], us.US_ERR_INVALID_ARG, [(0, 20)]),
            ([0, 0, 0, 0], [0, -1, 70, 130], us.US_ERR_INVALID_ARG, []),
            ([0, 0, 0, 0], [0, 40, 70, 130], us.US_OK, [])):
        o.fill_(7.0)
        us.us_attn_rows(dev(s.Q), dev(s.K), dev(s.R), dev(s.V), i32(off), i32(kv_off), 30, s.scale, o, ws)
        assert us.us_get_last_device_status() == code, (off, kv_off)
        for a, b in kept:
            assert np.array_equal(o[a:b].cpu().numpy(), good[a:b])
        assert (o[off[3]:] == 7).all()
