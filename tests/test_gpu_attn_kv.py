"""Attention over the quantised cache on the GPU against the plain 64-bit
reference.

Tolerance.  Codes and queries enter the products exactly; what is rounded is
the weight (fp16, relative 2^-11, of itself and once more through the V scale),
the output (fp16, 2^-11) and the fp32 score: its error is at most
(D + 8) 2^-24 of sum |q||k| scale, which moves a weight by that relative
amount (twice: the weight and the sum).  So with A = sum w|v| / sum w,
|err| <= 2^-11 |o| + A (2 2^-11 + 2 (D + 8) 2^-24 S) + a smallest fp16 step.
"""
import numpy as np
import pytest
import torch

from oracle import kv
from tests.test_gpu_kv_cache import dev, offsets, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


class Setup:
    """A cache filled with random history for requests of (ctx, n), NaN scales
    behind each request's last position, and query rows."""

    def __init__(self, us, elem, D, Hkv, G, page, ctx, n, seed, vspread=1.0):
        self.us, self.ctx, self.n = us, ctx, n
        rng = self.rng = np.random.default_rng(seed)
        need = [-(-max(c + k, 1) // page) for c, k in zip(ctx, n)]
        ids = rng.permutation(sum(need) + 1)
        table = np.full((len(ctx), max(need) + 1), -1, np.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = ids[at:at + k]
            at += k
        r = self.ref = kv.Cache(elem, D, Hkv, page, len(ids), table)
        for i, pool in enumerate((r.k, r.v)):
            x = rng.standard_normal((*pool.shape[:3], D))
            x *= np.exp(vspread * rng.standard_normal((*pool.shape[:3], 1)))
            c, s = kv.quantise(x.astype(np.float16), elem)
            pool[:], r.scale[..., i] = kv.pack(c, elem), s
        for b, (c, k) in enumerate(zip(ctx, n)):                # garbage behind the last position
            for p in range(c + k, need[b] * page):
                g, s = r.at(b, p)
                r.scale[g, :, s] = np.nan
        r.scale[ids[at]] = np.nan
        self.C = us.KVCache(elem, D, dev(r.k), dev(r.v), dev(r.scale), dev(table))
        self.T, self.Hq, self.D = sum(n), Hkv * G, D
        self.scale = D ** -0.5
        self.Q = (rng.standard_normal((self.T, self.Hq, D)) * 2).astype(np.float16)

    def tree(self, empty=()):
        """Random trees; tokens (by row) in `empty` see none of the call's tokens."""
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
        buf = torch.full((2, self.T, self.Hq * self.D + pad), 7.0, dtype=torch.float16, device="cuda")
        buf[0, :, :self.Hq * self.D] = dev(self.Q).reshape(self.T, -1)
        q, o = (x[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D)) for x in buf)
        max_n = max_n or max(self.n)
        ws = us.workspace_attn_kv(C, self.Hq, max_n) if ws is None else ws
        us.us_attn_kv(C, q, dev(offsets(self.n)), dev(np.array(self.ctx, np.int32)),
                      None if words is None else dev(words), max_n, self.scale, o, ws)
        assert us.us_get_last_device_status() == us.US_OK
        if pad:
            assert (buf[1, :, self.Hq * self.D:] == 7).all()
        return o.cpu().numpy().astype(np.float64)

    def check(self, got, grids, only=None):
        t = 0
        for b, k in enumerate(self.n):
            if only is None or b in only:
                want, mag, big = kv.attend(self.ref, b, self.Q[t:t + k], self.ctx[b], grids[b], self.scale)
                tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -24
                       + mag * (2 * 2.0 ** -11 + 2 * (self.D + 8) * 2.0 ** -24 * big[..., None]))
                err = np.abs(got[t:t + k] - want)
                assert np.isfinite(got[t:t + k]).all()
                assert (err <= tol).all(), f"request {b}: {np.max(err / tol):.2f} times the tolerance"
            t += k


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,G,page,ctx", [
    (128, 8, 4, 16, [777]),
    (128, 1, 1, 64, [0, 1, 15, 16, 17, 63, 64, 65, 130]),
    (64, 2, 7, 16, [300, 5, 0, 1023]),
    (128, 2, 8, 32, [2500, 31, 200]),
    (64, 1, 16, 128, [511, 90]),
    (128, 1, 32, 64, [700, 0, 33]),
    (64, 1, 48, 64, [259]),
])
def test_single_tokens(us, elem, D, Hkv, G, page, ctx):
    s = Setup(us, elem, D, Hkv, G, page, ctx, [1] * len(ctx), 11)
    words, grids = s.tree()
    got = s.run(words, pad=16)
    s.check(got, grids)
    assert np.array_equal(got, s.run(None))                    # a chain of one is a tree of one


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,Hkv,G,page,ctx,n", [
    (128, 2, 4, 64, [200, 0, 63], [64, 64, 1]),
    (64, 4, 1, 32, [100, 7, 450, 0], [13, 25, 0, 2]),
    (128, 1, 5, 16, [33, 129], [7, 50]),
    (128, 2, 1, 16, [1200], [5]),
    (64, 1, 8, 128, [77, 1, 300], [33, 64, 3]),
    (128, 1, 8, 64, [500], [64]),
])
def test_trees(us, elem, D, Hkv, G, page, ctx, n):
    s = Setup(us, elem, D, Hkv, G, page, ctx, n, 12)
    words, grids = s.tree()
    s.check(s.run(words, max_n=64, pad=8), grids)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("D,G,ctx,n", [
    (128, 4, [100, 0], [70, 129]), (64, 1, [0], [300]), (128, 1, [31, 5, 250], [2, 150, 1]), (128, 8, [127], [65])])
def test_chains(us, elem, D, G, ctx, n):
    s = Setup(us, elem, D, 1, G, 32, ctx, n, 13)
    words, grids = s.chain()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("G,n", [(4, 3), (4, 20), (1, 64)])
def test_rows_that_see_nothing(us, G, n):
    """Rows with an empty mask: the context alone, or nothing at all (output 0)."""
    s = Setup(us, kv.I8, 128, 2, G, 16, [0, 40], [n, n], 14)
    words, grids = s.tree(empty={0, n - 1, n, 2 * n - 1})
    got = s.run(words)
    s.check(got, grids)
    assert (got[0] == 0).all() and (got[n - 1] == 0).all() and (got[n] != 0).any()


@pytest.mark.parametrize("G,n", [(2, 5), (8, 64)])
def test_mask_bits_behind_the_tokens_are_ignored(us, G, n):
    s = Setup(us, kv.I4, 64, 1, G, 16, [50, 9], [n, 3], 15)
    words, grids = s.tree()
    more = words.copy()
    more[n:] |= np.int64(-8)                                    # bits 3..63 of the second request's words
    assert np.array_equal(s.run(words, max_n=64), s.run(more, max_n=64))
    s.check(s.run(more, max_n=64), grids)


@pytest.mark.parametrize("elem", [kv.I8, kv.I4])
@pytest.mark.parametrize("G,n", [(4, 1), (1, 12), (4, 40)])
def test_values_of_very_different_scales(us, elem, G, n):
    """V rows whose magnitudes spread over e^+-12 and sharp scores."""
    s = Setup(us, elem, 128, 1, G, 64, [333], [n], 16, vspread=3.0)
    words, grids = s.tree()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("vscale", [2.0 ** -24, 2.0 ** -14, 60000.0])
@pytest.mark.parametrize("G,n", [(4, 1), (4, 32)])
def test_smallest_and_largest_value_scales(us, vscale, G, n):
    s = Setup(us, kv.I8, 64, 1, G, 16, [100], [n], 17, vspread=0.0)
    c = np.clip(kv.unpack(s.ref.v, kv.I8), -1, 1)
    s.ref.v[:] = kv.pack(c, kv.I8)
    fin = np.isfinite(s.ref.scale[..., 1].astype(np.float32))
    s.ref.scale[..., 1][fin] = vscale
    s.C = us.KVCache(kv.I8, 64, s.C.k, dev(s.ref.v), dev(s.ref.scale), s.C.page_table)
    words, grids = s.tree()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("G,n", [(4, 1), (4, 9), (8, 64)])
def test_nan_in_unseen_entries(us, G, n):
    """Drafted entries that a row does not see may hold anything."""
    s = Setup(us, kv.I8, 128, 1, G, 16, [90], [n], 18)
    words, grids = s.tree()
    words[:] &= ~np.int64(1 << (n - 1)) if n < 64 else np.int64(2 ** 63 - 1)
    for g in grids[0]:
        g[n - 1] = 0
    got = s.run(words)
    g, slot = s.ref.at(0, 90 + n - 1)
    s.C.scale[g, :, slot] = float("nan")
    assert np.array_equal(got, s.run(words))
    s.ref.scale[g, :, slot] = 0
    s.check(got, grids)


def test_many_requests_and_repeatability(us):
    """More requests than SMs, lengths from nothing to long, the same bits twice, one workspace for all calls."""
    rng = np.random.default_rng(19)
    ctx = [int(x) for x in np.exp(rng.uniform(0, 7.5, 300))]
    s = Setup(us, kv.I4, 64, 2, 4, 16, ctx, [1] * 300, 20)
    words, grids = s.tree()
    ws = us.workspace_attn_kv(s.C, s.Hq, 64)
    got = s.run(words, ws=ws)
    s.check(got, grids, only=set(range(0, 300, 9)) | {int(np.argmax(ctx))})
    for _ in range(3):
        assert np.array_equal(got, s.run(words, ws=ws))
    s.check(s.run(words, max_n=64, ws=ws), grids, only={0, 7, 299})
    assert np.array_equal(got, s.run(words, ws=ws))


@pytest.mark.parametrize("G,n", [(4, 1), (4, 16)])
def test_long_context(us, G, n):
    """A context that one request's many partial results are joined over; a constant V gives that constant."""
    ctx = 40000
    s = Setup(us, kv.I8, 64, 1, G, 64, [ctx], [n], 21)
    s.ref.v[:] = 50
    s.ref.scale[..., 1] = np.where(np.isnan(s.ref.scale[..., 1]), s.ref.scale[..., 1], np.float16(0.25))
    s.C = us.KVCache(kv.I8, 64, s.C.k, dev(s.ref.v), dev(s.ref.scale), s.C.page_table)
    got = s.run(s.tree()[0])
    assert np.abs(got - 12.5).max() <= 12.5 * 3 * 2.0 ** -11


def test_queries_in_a_fused_row_and_another_stream(us):
    s = Setup(us, kv.I8, 128, 2, 4, 64, [300, 20], [1, 1], 22)
    words, grids = s.tree()
    want = s.run(words)
    fused = torch.zeros(2, 8 * 128 + 4 * 128, dtype=torch.float16, device="cuda")
    q = fused[:, :1024].unflatten(1, (8, 128))
    out = torch.zeros(2, 8, 128, dtype=torch.float16, device="cuda")
    ws = us.workspace_attn_kv(s.C, 8, 1)
    off, pos, m = dev(offsets([1, 1])), dev(np.array([300, 20], np.int32)), dev(words)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.copy_(dev(s.Q))
        us.us_attn_kv(s.C, q, off, pos, m, 1, s.scale, out, ws)
    side.synchronize()
    assert np.array_equal(out.cpu().numpy().astype(np.float64), want)


def test_captured_graph_follows_lengths(us):
    s = Setup(us, kv.I4, 128, 2, 4, 16, [900], [1], 23)
    words, grids = s.tree()
    ws = us.workspace_attn_kv(s.C, s.Hq, 1)
    q, m, off = dev(s.Q), dev(words), dev(offsets([1]))
    pos, out = dev(np.array([900], np.int32)), torch.zeros(1, s.Hq, 128, dtype=torch.float16, device="cuda")
    us.us_attn_kv(s.C, q, off, pos, m, 1, s.scale, out, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        us.us_attn_kv(s.C, q, off, pos, m, 1, s.scale, out, ws)
    for ctx in (0, 5, 640, 900):
        pos.fill_(ctx)
        graph.replay()
        s.ctx = [ctx]
        s.check(out.cpu().numpy().astype(np.float64), grids)


def test_bad_lengths_and_pages_are_recorded(us):
    s = Setup(us, kv.I8, 64, 1, 2, 16, [40, 60], [1, 1], 24)
    words, grids = s.tree()
    ws = us.workspace_attn_kv(s.C, s.Hq, 1)
    out = torch.full((2, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    args = (dev(s.Q), dev(offsets([1, 1])))
    for pos in ([-1, 60], [2**31 - 1, 60], [16 * s.C.page_table.shape[1], 60]):
        out.fill_(7.0)
        us.us_attn_kv(s.C, *args, dev(np.array(pos, np.int32)), dev(words), 1, s.scale, out, ws)
        assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
        assert (out[0] == 7).all()
        s.check(out.cpu().numpy().astype(np.float64), grids, only={1})
    s.C.page_table[0, 1] = -1                                   # positions 16..31 are not attended to
    us.us_attn_kv(s.C, *args, dev(np.array([40, 60], np.int32)), dev(words), 1, s.scale, out, ws)
    assert us.us_get_last_device_status() == us.US_ERR_CORRUPT
    got = out.cpu().numpy().astype(np.float64)
    s.check(got, grids, only={1})
    s.ref.table = s.ref.table.copy()
    s.ref.table[0, 1:-1], s.ref.table[0, -1] = s.ref.table[0, 2:], -1
    s.ctx[0] = 24
    s.check(got, grids, only={0})


@pytest.mark.parametrize("elem,D,G,n", [(kv.I4, 64, 1, 64), (kv.I8, 128, 4, 40), (kv.I8, 128, 4, 6), (kv.I4, 64, 3, 9)])
def test_states_of_many_ctas(us, elem, D, G, n):
    """One request whose tiles go to a CTA each: two dozen or more partial states a row."""
    s = Setup(us, elem, D, 1, G, 64, [2900], [n], 25)
    words, grids = s.tree()
    s.check(s.run(words), grids)


@pytest.mark.parametrize("D,G,n", [(128, 4, 1), (128, 4, 6), (64, 4, 8), (64, 4, 16), (128, 4, 40)])
def test_scores_that_rise_along_the_context(us, D, G, n):
    """Keys that grow tile after tile: the largest score moves all the way, and with it what came before."""
    s = Setup(us, kv.I8, D, 2, G, 32, [900, 50], [n, n], 26)
    for b, (c, k) in enumerate(zip(s.ctx, s.n)):
        for p in range(c + k):
            g, slot = s.ref.at(b, p)
            s.ref.scale[g, :, slot, 0] *= np.float16(0.25 + p / 50)
    s.C = us.KVCache(kv.I8, D, s.C.k, s.C.v, dev(s.ref.scale), s.C.page_table)
    words, grids = s.tree()
    s.check(s.run(words), grids)
