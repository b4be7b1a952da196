"""Attention over latent rows on the GPU against the plain 64-bit reference.

Tolerance.  Rows and queries enter the products exactly.  A weight is rounded to fp16
(2^-11 of itself) and the output (2^-11).  The fp32 score is off by at most (W + 8) 2^-24
of S = sum |q||x| scale, which moves a weight, and their sum, by that.  Sums and outputs
are accumulated in fp32 over L positions, in no more than L / 8 steps each: L 2^-26 in
all.  Weights below fp16's normal range are off by 2^-25 where the largest is 2^11:
L 2^-36 of the largest value, within the last term for these lengths.
|err| <= 2^-11 |o| + A (2^-11 + 2 (W + 8) 2^-24 S + L 2^-26) + 2^-24 max|x|,  A = sum w|x|."""
import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_gpu_kv_cache import dev, offsets
from tests.test_gpu_rope import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


class Setup:
    """Random rows for requests of (ctx, n), NaN behind each one's last position and in the spare page."""

    def __init__(self, us, Dc, Hq, page, ctx, n, seed, spread=0.0, sharp=1.0):
        self.us, self.ctx, self.n, self.Dc, self.Hq = us, ctx, n, Dc, Hq
        rng = self.rng = np.random.default_rng(seed)
        W = self.W = Dc + 64
        need = [-(-max(c + k, 1) // page) for c, k in zip(ctx, n)]
        ids = rng.permutation(sum(need) + 1)
        self.table = np.full((len(ctx), max(need) + 1), -1, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = ids[sum(need[:b]):sum(need[:b + 1])]
        pool = rng.standard_normal((len(ids), page, W)) * np.exp(spread * rng.standard_normal((len(ids), page, 1)))
        self.pool = pool.astype(np.float16)
        for b, (c, k) in enumerate(zip(ctx, n)):
            for p in range(c + k, need[b] * page):
                self.pool[self.table[b, p // page], p % page] = np.nan
        self.pool[ids[-1]] = np.nan
        self.page, self.T, self.scale = page, sum(n), W ** -0.5
        self.Q = (sharp * rng.standard_normal((self.T, Hq, W))).astype(np.float16)
        self.load()

    def load(self):
        self.C = self.us.LatCache(self.Dc, 64, dev(self.pool), dev(self.table))

    def rows(self, b):
        m = -(-(self.ctx[b] + self.n[b]) // self.page)
        return self.pool[self.table[b, :m]].reshape(-1, self.W)[:self.ctx[b] + self.n[b]]

    def tree(self, empty=()):
        words, grids, t = [], [], 0
        for k in self.n:
            of = []
            for i in range(k):
                of.append((of[self.rng.integers(0, i)] if i and self.rng.random() < 0.9 else 0) | 1 << i)
            of = [0 if t + i in empty else m for i, m in enumerate(of)]
            grids.append([[m >> j & 1 for j in range(k)] for m in of])
            words += of
            t += k
        return np.array([m - (1 << 64) if m >> 63 else m for m in words], np.int64), grids

    def chain(self):
        return None, [[[j <= i for j in range(k)] for i in range(k)] for k in self.n]

    def run(self, words, max_n=None, pad=0, ws=None):
        us, C = self.us, self.C
        q = torch.full((self.T + 1, self.Hq * self.W + pad), 7.0, dtype=torch.float16, device="cuda")
        o = torch.full((self.T + 1, self.Hq * self.Dc + pad), 7.0, dtype=torch.float16, device="cuda")
        q[:self.T, :self.Hq * self.W] = dev(self.Q).reshape(self.T, -1)
        max_n = max_n or max(self.n)
        ws = us.workspace_attn_lat(C, self.Hq, max_n) if ws is None else ws
        qv, ov = q[:self.T, :self.Hq * self.W].unflatten(1, (self.Hq, self.W)), o[:self.T, :self.Hq * self.Dc].unflatten(1, (self.Hq, self.Dc))
        us.us_attn_lat(C, qv, dev(offsets(self.n)), i32(self.ctx), None if words is None else dev(words), max_n, self.scale, ov, ws)
        assert us.us_get_last_device_status() == us.US_OK
        assert (o[self.T] == 7).all() and (o[:, self.Hq * self.Dc:] == 7).all()
        return ov.cpu().numpy().astype(np.float64)

    def check(self, got, grids, only=None):
        t = 0
        for b, k in enumerate(self.n):
            if only is None or b in only:
                x, L = self.rows(b), self.ctx[b] + k
                seen = np.ones((k, L), bool)
                if k:
                    seen[:, self.ctx[b]:] = np.array(grids[b], bool).reshape(k, k)
                q = self.Q[t:t + k].reshape(k * self.Hq, self.W)
                want, mag, big = lat.attend(q, x, x[:, :self.Dc], np.repeat(seen, self.Hq, 0), self.scale)
                most = np.abs(np.nan_to_num(x.astype(np.float64), nan=0, posinf=0, neginf=0)).max() if L else 0
                tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -24 * most
                       + mag * (2.0 ** -11 + 2 * (self.W + 8) * 2.0 ** -24 * big[:, None] + L * 2.0 ** -26))
                err = np.abs(got[t:t + k].reshape(k * self.Hq, self.Dc) - want)
                assert np.isfinite(got[t:t + k]).all()
                assert (err <= tol).all(), f"request {b}: {np.max(err / tol):.2f} times the tolerance"
            t += k


@pytest.mark.parametrize("Dc,Hq,page,ctx", [
    (512, 16, 16, [777]),
    (512, 32, 64, [0, 1, 15, 16, 17, 63, 64, 65, 130]),
    (256, 8, 16, [300, 5, 0, 1023]),
    (512, 64, 32, [2500, 31, 200]),
    (256, 128, 128, [511, 90]),
    (512, 1, 64, [700, 0, 33]),
    (512, 20, 16, [259, 64]),
    (256, 65, 1024, [1500]),
    (512, 128, 64, [127, 128]),
])
def test_single_tokens(us, Dc, Hq, page, ctx):
    s = Setup(us, Dc, Hq, page, ctx, [1] * len(ctx), 11)
    words, grids = s.tree()
    got = s.run(words, pad=16)
    s.check(got, grids)
    assert np.array_equal(got, s.run(None))                    # a chain of one is a tree of one


@pytest.mark.parametrize("Dc,Hq,n", [(256, 64, 1), (512, 64, 1), (512, 16, 4), (256, 20, 9)])
def test_many_segments_a_cta(us, Dc, Hq, n):
    """Several requests' tiles on every SM, of one to ten tiles each."""
    ctx = [int(c) for c in np.random.default_rng(21).integers(0, 600, 170)]
    s = Setup(us, Dc, Hq, 64, ctx, [n] * len(ctx), 22)
    words, grids = s.tree()
    ws = us.workspace_attn_lat(s.C, Hq, n)
    got = s.run(words, ws=ws)
    s.check(got, grids, only=range(0, len(ctx), 7))
    for _ in range(3):
        assert np.array_equal(got, s.run(words, ws=ws))


@pytest.mark.parametrize("Dc,Hq,page,ctx,n", [
    (512, 16, 64, [200, 0, 63], [64, 64, 1]),
    (256, 4, 32, [100, 7, 450, 0], [13, 25, 0, 2]),
    (512, 20, 16, [33, 129], [7, 50]),
    (512, 32, 16, [1200], [5]),
    (256, 64, 128, [77, 1, 300], [3, 5, 3]),
    (512, 1, 64, [500], [64]),
    (512, 7, 16, [10, 100], [9, 10]),
])
def test_trees(us, Dc, Hq, page, ctx, n):
    s = Setup(us, Dc, Hq, page, ctx, n, 12)
    words, grids = s.tree()
    s.check(s.run(words, max_n=64, pad=8), grids)


@pytest.mark.parametrize("Dc,Hq,ctx,n", [(512, 4, [100, 0], [70, 129]), (256, 1, [0], [300]), (512, 3, [31, 5, 250], [2, 150, 1]), (256, 64, [127], [11])])
def test_chains(us, Dc, Hq, ctx, n):
    s = Setup(us, Dc, Hq, 32, ctx, n, 13)
    words, grids = s.chain()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("Hq,n", [(4, 3), (16, 20), (1, 64)])
def test_rows_that_see_nothing(us, Hq, n):
    s = Setup(us, 512, Hq, 16, [0, 40], [n, n], 14)
    words, grids = s.tree(empty={0, n - 1, n, 2 * n - 1})
    got = s.run(words)
    s.check(got, grids)
    assert (got[0] == 0).all() and (got[n - 1] == 0).all() and (got[n] != 0).any()


@pytest.mark.parametrize("n", [5, 64])
def test_mask_bits_behind_the_tokens_are_ignored(us, n):
    s = Setup(us, 256, 8, 16, [50, 9], [n, 3], 15)
    words, grids = s.tree()
    more = words.copy()
    more[n:] |= np.int64(-8)
    assert np.array_equal(s.run(words, max_n=64), s.run(more, max_n=64))
    s.check(s.run(more, max_n=64), grids)


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("Dc,Hq,n", [(512, 4, 9), (256, 16, 64), (512, 64, 2)])
def test_unseen_entries_may_hold_anything(us, what, Dc, Hq, n):
    s = Setup(us, Dc, Hq, 16, [90], [n], 18)
    words, grids = s.tree()
    words &= ~np.int64(1 << (n - 1)) if n < 64 else np.int64(2 ** 63 - 1)
    for g in grids[0]:
        g[n - 1] = 0
    s.pool[s.table[0, (90 + n - 1) // 16], (90 + n - 1) % 16] = what
    s.load()
    s.check(s.run(words), grids)


def test_rows_that_see_what_is_not_finite_are_nan(us):
    s = Setup(us, 512, 4, 16, [20], [6], 19)
    words, grids = s.chain()
    s.pool[s.table[0, 1], 8, 100] = np.nan                     # position 24, the call's fifth
    s.load()
    got = s.run(words)
    assert np.isfinite(got[:4]).all() and np.isnan(got[4:]).all()


@pytest.mark.parametrize("Hq,n", [(16, 1), (4, 12), (64, 4)])
def test_values_of_very_different_sizes(us, Hq, n):
    s = Setup(us, 512, Hq, 64, [333], [n], 16, spread=1.5, sharp=0.3)
    words, grids = s.tree()
    s.check(s.run(words), grids)


def test_scores_that_rise_along_the_context(us):
    """References move tile after tile, and between the CTAs that share a request."""
    s = Setup(us, 256, 16, 16, [1500], [1], 20)
    ramp = np.linspace(-40, 40, s.pool.shape[0] * 16)
    for p in range(1501):
        s.pool[s.table[0, p // 16], p % 16, 256:] = 0
        s.pool[s.table[0, p // 16], p % 16, 256] = ramp[p]
    s.Q[..., 256] = 20.0
    s.load()
    words, grids = s.tree()
    s.check(s.run(words), grids)
    s.Q[..., 256] = -20.0
    s.check(s.run(words), grids)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-6])
def test_scales(us, scale):
    s = Setup(us, 512, 8, 64, [150, 3], [3, 3], 21)
    s.scale = scale
    words, grids = s.tree()
    s.check(s.run(words), grids)


def test_many_requests_and_repeatability(us):
    """More requests than SMs, lengths from nothing to long, the same bits twice, one workspace for all calls."""
    rng = np.random.default_rng(19)
    ctx = [int(x) for x in np.exp(rng.uniform(0, 7, 300))]
    s = Setup(us, 256, 12, 16, ctx, [1] * 300, 22)
    words, grids = s.tree()
    ws = us.workspace_attn_lat(s.C, s.Hq, 64)
    got = s.run(words, ws=ws)
    s.check(got, grids, only=set(range(0, 300, 9)) | {int(np.argmax(ctx))})
    for _ in range(3):
        assert np.array_equal(got, s.run(words, ws=ws))
    s.check(s.run(words, max_n=64, ws=ws), grids, only={0, 7, 299})
    assert np.array_equal(got, s.run(words, ws=ws))


@pytest.mark.parametrize("Hq,n", [(16, 1), (4, 16)])
def test_long_context(us, Hq, n):
    """One request's many partial states joined; a constant value gives that constant."""
    s = Setup(us, 256, Hq, 64, [40000], [n], 23)
    fin = np.isfinite(s.pool[..., 0].astype(np.float32))
    s.pool[fin, :256] = 12.5
    s.load()
    got = s.run(s.tree()[0])
    assert np.abs(got - 12.5).max() <= 12.5 * (3 * 2.0 ** -11 + 40000 * 2.0 ** -26)


def test_bad_requests_are_skipped(us):
    s = Setup(us, 512, 4, 16, [40, 10, 30], [2, 3, 4], 24)
    words, grids = s.chain()
    o = torch.full((9, 4, 512), 7.0, dtype=torch.float16, device="cuda")
    ws = us.workspace_attn_lat(s.C, 4, 4)
    q = dev(s.Q)
    us.us_attn_lat(s.C, q, i32([0, 2, 5, 9]), i32([40, 16 * s.table.shape[1] - 2, 30]), None, 4, s.scale, o, ws)
    assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
    assert (o[2:5] == 7).all()
    s.check(np.nan_to_num(o.cpu().numpy().astype(np.float64)), grids, only={0, 2})
    s.C.page_table[0, 1] = 12345                               # 16 positions that are not attended to
    us.us_attn_lat(s.C, q, i32([0, 2, 5, 9]), i32(s.ctx), None, 4, s.scale, o, ws)
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    x = np.delete(s.rows(0), np.s_[16:32], 0)
    want, mag, big = lat.attend(s.Q[1], x, x[:, :512], np.ones((4, len(x)), bool), s.scale)
    assert np.abs(o[1].cpu().numpy() - want).max() <= 2e-3 * np.abs(x.astype(np.float64)).max()
    s.check(o.cpu().numpy().astype(np.float64), grids, only={1, 2})


def test_another_stream_and_two_graphs(us):
    """A call on a side stream; two captured graphs of their own workspaces, replayed in turn and together."""
    s, t = Setup(us, 512, 16, 64, [300, 20], [1, 1], 25), Setup(us, 256, 32, 16, [90], [7], 26)
    out = []
    for x in (s, t):
        words, grids = x.tree()
        want = x.run(words)
        x.check(want, grids)
        q, o = dev(x.Q), torch.zeros(x.T, x.Hq, x.Dc, dtype=torch.float16, device="cuda")
        off, pos, m, ws = dev(offsets(x.n)), i32(x.ctx), dev(words), us.workspace_attn_lat(x.C, x.Hq, max(x.n))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call = lambda x=x, q=q, o=o, off=off, pos=pos, m=m, ws=ws: us.us_attn_lat(x.C, q, off, pos, m, max(x.n), x.scale, o, ws)  # noqa: E731
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert np.array_equal(o.cpu().numpy(), want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        out.append((g, o, want, side, call))                   # (the call's tensors live as long as the graph)
    for _ in range(3):
        for g, o, want, side, _ in out:
            o.zero_()
        torch.cuda.synchronize()
        for g, o, want, side, _ in out:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for g, o, want, side, _ in out:
            assert np.array_equal(o.cpu().numpy(), want)
    assert us.us_get_last_device_status() == us.US_OK
