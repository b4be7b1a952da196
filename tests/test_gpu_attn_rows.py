"""Causal attention over expanded rows on the GPU against the plain 64-bit reference.
Tolerance as for the attention over latent rows, with W = Dn + 64 and values V."""
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
    def __init__(self, us, D, H, kv, n, seed, spread=0.0, sharp=1.0):
        """kv: key rows a request (None: n of them), n: query rows."""
        self.us, self.D, self.H, self.n = us, D, H, n
        self.kv = kv
        rng = self.rng = np.random.default_rng(seed)
        self.T, self.S, self.scale = sum(n), sum(kv), (D + 64) ** -0.5
        f = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.Q = (sharp * f(self.T, H, D + 64)).astype(np.float16)
        self.K, self.R = f(self.S, H, D).astype(np.float16), f(self.S, 64).astype(np.float16)
        self.V = (f(self.S, H, D) * np.exp(spread * f(self.S, 1, 1))).astype(np.float16)

    def run(self, max_n=None, ws=None, side_by_side=True, gap=0):
        us, H, D, S, T = self.us, self.H, self.D, self.S, self.T
        if side_by_side:                                       # as one expansion gives them
            both = torch.full((S, H, 2 * D + gap), float("nan"), dtype=torch.float16, device="cuda")
            both[..., :D], both[..., D:2 * D] = dev(self.K), dev(self.V)
            k, v = both[..., :D], both[..., D:2 * D]
        else:
            k, v = dev(self.K), dev(self.V)
        kr = torch.full((S, 64 + 8 + gap), float("nan"), dtype=torch.float16, device="cuda")
        kr[:, 8:72] = dev(self.R)
        q = torch.full((T, H * (D + 64) + gap), 7.0, dtype=torch.float16, device="cuda")
        q[:, :H * (D + 64)] = dev(self.Q).reshape(T, -1)
        o = torch.full((T + 1, H * D + gap), 7.0, dtype=torch.float16, device="cuda")
        max_n = max_n or max(self.n)
        ws = us.workspace_attn_rows(D, 64, D, H, len(self.n), max_n) if ws is None else ws
        ov = o[:T, :H * D].unflatten(1, (H, D))
        us.us_attn_rows(q[:, :H * (D + 64)].unflatten(1, (H, D + 64)), k, kr[:, 8:72], v, dev(offsets(self.n)), dev(offsets(self.kv)),
                        max_n, self.scale, ov, ws)
        assert us.us_get_last_device_status() == us.US_OK
        assert (o[T] == 7).all() and (o[:, H * D:] == 7).all()
        return ov.cpu().numpy().astype(np.float64)

    def check(self, got, only=None, heads=None):
        t = s = 0
        for b, (k, L) in enumerate(zip(self.n, self.kv)):
            if only is None or b in only:
                seen = np.tril(np.ones((k, L), bool), L - k)
                for h in heads if heads is not None else range(self.H):
                    key = np.concatenate((self.K[s:s + L, h], self.R[s:s + L]), 1)
                    val = self.V[s:s + L, h]
                    want, mag, big = lat.attend(self.Q[t:t + k, h], key, val, seen, self.scale)
                    most = np.abs(np.nan_to_num(val.astype(np.float64), nan=0, posinf=0, neginf=0)).max(initial=0)
                    tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -24 * most
                           + mag * (2.0 ** -11 + 2 * (self.D + 72) * 2.0 ** -24 * big[:, None] + L * 2.0 ** -26))
                    err = np.abs(got[t:t + k, h] - want)
                    assert np.isfinite(got[t:t + k, h]).all()
                    assert (err <= tol).all(), f"request {b} head {h}: {np.max(err / tol):.2f} times the tolerance"
            t, s = t + k, s + L


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("H,kv,n", [
    (1, [1], [1]), (2, [5, 1, 0, 129], [5, 1, 0, 129]), (1, [128], [128]), (3, [127, 256, 257], [127, 256, 257]),
    (2, [700], [700]), (4, [1000, 90, 300], [1, 90, 3]), (1, [1500], [400]), (5, [130, 131], [129, 2]),
    (2, [385, 640, 513], [256, 384, 512]), (8, [33] * 40, [33] * 40), (1, [64, 0, 4000], [64, 0, 1]),
])
def test_against_the_reference(us, D, H, kv, n):
    s = Setup(us, D, H, kv, n, D + H)
    got = s.run()
    s.check(got)
    assert np.array_equal(got, s.run(side_by_side=False, gap=16))
    s.check(s.run(max_n=max(n) + 300))                         # (another max_n may join states in another order)


def test_long_prompts_on_many_heads(us):
    """More segments than SMs, whole ones and shared ones."""
    s = Setup(us, 128, 20, [1300, 2100, 700], [1300, 300, 700], 1)
    got = s.run()
    s.check(got, heads=[0, 7, 19])
    ws = us.workspace_attn_rows(128, 64, 128, 20, 3, 1300)
    for _ in range(3):
        assert np.array_equal(got, s.run(ws=ws))


@pytest.mark.parametrize("D", [128, 64])
def test_many_short_segments(us, D):
    """Several segments on every SM, of which the two streams read unlike numbers of tiles."""
    n = [20, 300, 1, 140, 256, 40] * 4
    kv = [20, 300, 129, 260, 500, 41] * 4
    s = Setup(us, D, 40, kv, n, 5)
    ws = us.workspace_attn_rows(D, 64, D, 40, len(n), 300)
    got = s.run(ws=ws)
    s.check(got, heads=[0, 13, 39])
    for _ in range(3):
        assert np.array_equal(got, s.run(ws=ws))


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-6])
def test_scales(us, scale):
    s = Setup(us, 128, 2, [300, 20], [200, 20], 2)
    s.scale = scale
    s.check(s.run())


def test_scores_that_rise_along_the_keys(us):
    for sign in (20.0, -20.0):
        s = Setup(us, 64, 2, [1500], [300], 3)
        s.R[:] = 0
        s.R[:, 0] = np.linspace(-40, 40, 1500)
        s.Q[..., 64] = sign
        s.check(s.run())


def test_values_of_very_different_sizes(us):
    s = Setup(us, 128, 2, [500], [500], 4, spread=2.0)
    s.check(s.run())


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("n", [150, 300, 512])
def test_later_rows_may_hold_anything(us, what, n):
    """Values and keys that a query does not see, in its own request and in the next one."""
    s = Setup(us, 128, 2, [n, 40], [n, 40], 5)
    whole = s.run()
    s.check(whole)
    cut = n - 30
    for x in (s.K, s.V, s.R):
        x[cut:n] = what
    got = s.run()
    assert np.array_equal(got[:cut], whole[:cut]) and np.array_equal(got[n:], whole[n:])
    assert np.isnan(got[cut:n]).all()


def test_bad_requests_are_skipped(us):
    s = Setup(us, 64, 2, [40, 50, 60], [10, 20, 60], 6)
    o = torch.full((90, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    args = dev(s.Q), dev(s.K), dev(s.R), dev(s.V)
    ws = us.workspace_attn_rows(64, 64, 64, 2, 3, 60)
    good = s.run()
    same, skipped = slice, slice
    for kv_off, off, kept, left in (
            ([0, 40, 45, 105], [0, 10, 30, 90], same(0, 10), skipped(10, 30)),      # more queries than keys
            ([0, 40, 90, 151], [0, 10, 30, 90], same(0, 30), skipped(30, 90)),      # beyond the key rows
            ([0, 40, 30, 150], [0, 10, 30, 90], same(0, 10), skipped(10, 30)),      # descending
            ([-1, 40, 90, 150], [0, 10, 30, 90], same(10, 90), skipped(0, 10)),
            ([0, 40, 90, 150], [0, 10, 5, 90], same(0, 10), skipped(10, 90))):      # the last one then has more than max_n
        o.fill_(7.0)
        us.us_attn_rows(*args, i32(off), i32(kv_off), 60, s.scale, o, ws)
        assert us.us_get_last_device_status() == us.US_ERR_INVALID_ARG
        got = o.cpu().numpy()
        assert np.array_equal(got[kept], good[kept]) and (got[left] == 7).all()
    us.us_attn_rows(*args, i32([0, 10, 30, 90]), i32([0, 40, 90, 150]), 60, s.scale, o, ws)
    assert us.us_get_last_device_status() == us.US_OK and np.array_equal(o.cpu().numpy(), good)


def test_another_stream_and_a_graph(us):
    s = Setup(us, 128, 4, [700, 300], [300, 300], 7)
    want = s.run()
    args = dev(s.Q), dev(s.K), dev(s.R), dev(s.V), dev(offsets(s.n)), dev(offsets(s.kv)), 300, s.scale
    o, ws = torch.zeros(600, 4, 128, dtype=torch.float16, device="cuda"), us.workspace_attn_rows(128, 64, 128, 4, 2, 300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        us.us_attn_rows(*args, o, ws)
    side.synchronize()
    assert np.array_equal(o.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        us.us_attn_rows(*args, o, ws)
    for _ in range(3):
        o.zero_()
        g.replay()
        assert np.array_equal(o.cpu().numpy(), want)
    # the graph follows the offsets' values
    args[4].copy_(i32([0, 100, 400]))
    args[5].copy_(i32([0, 500, 1000]))
    g.replay()
    t = Setup(us, 128, 4, [500, 500], [100, 300], 7)
    t.Q, t.K, t.R, t.V, t.T, t.S = s.Q[:400], s.K, s.R, s.V, 400, 1000
    t.check(o[:400].cpu().numpy().astype(np.float64))
    assert us.us_get_last_device_status() == us.US_OK
