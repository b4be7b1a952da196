"""Drafted trees over latent rows from draft to commit, as a decoder uses the calls: pages, rotation by depth, the
write, attention under masks, the accepted path's rows moved, what is left of the pages given back."""
import numpy as np
import pytest
import torch

from oracle import lat
from tests.test_gpu_kv_cache import dev, offsets
from tests.test_gpu_rope import i32, rope, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


def tree(rng, n):
    """Words, depths and parents of n drafts, the first of them the root."""
    parent = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
    words, depth = [], []
    for i, p in enumerate(parent):
        words.append((words[p] if i else 0) | 1 << i)
        depth.append(depth[p] + 1 if i else 0)
    return words, depth, parent


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("Dc,Hq,page,start", [(512, 16, 16, [37, 0, 130]), (256, 64, 64, [300, 63, 64])])
def test_steps_of_drafted_trees(us, Dc, Hq, page, start, style):
    """Against the formulas, and, bit for bit, against a cache in which the accepted tokens were written one after the
    other: rows that were drafted at their depth and moved are the rows of a chain."""
    rng = np.random.default_rng(51)
    B, W = len(start), Dc + 64
    r = rope(us, 64, style)
    w = dev((1 + 0.3 * rng.standard_normal(Dc)).astype(np.float16))
    pools = [us.kv_pool(page, 80, B, 40) for _ in range(2)]
    drafted, chain = (us.lat_cache(Dc, 64, page, 80, p.page_table) for p in pools)
    drafted.rows.fill_(float("nan"))
    chain.rows.fill_(float("nan"))
    x = dev(values(rng, sum(start), 1, W)[:, 0])
    for p, C in zip(pools, (drafted, chain)):
        us.us_kv_reserve(p, i32(start))
        us.us_lat_write(C, r, x, w, dev(offsets(start)), i32([0] * B), None, max(start))
    length, scale = list(start), W ** -0.5
    ws = us.workspace_attn_lat(drafted, Hq, 64)
    for step in range(4):
        n = [int(v) for v in rng.integers(1, 65, B)]
        trees = [tree(rng, m) for m in n]
        depth = i32(sum((t[1] for t in trees), []))
        mask = dev(np.array([m - (1 << 64) if m >> 63 else m for t in trees for m in t[0]], np.int64))
        x, q = (values(rng, sum(n), h, W) for h in (1, Hq))
        x, q = dev(x[:, 0]), dev(q)
        off, pos = dev(offsets(n)), i32(length)
        us.us_kv_reserve(pools[0], i32([a + b for a, b in zip(length, n)]))
        part = q[..., Dc:]
        us.us_norm_rope(r, part, None, part, None, None, None, off, pos, depth, 64)
        us.us_lat_write(drafted, r, x, w, off, pos, depth, 64)
        o = torch.full((sum(n), Hq, Dc), 7.0, dtype=torch.float16, device="cuda")
        us.us_attn_lat(drafted, q, off, pos, mask, 64, scale, o, ws)
        # against the definition over the rows that are stored
        rows = torch.empty(sum(length) + sum(n), W, dtype=torch.float16, device="cuda")
        both = [a + b for a, b in zip(length, n)]
        us.us_lat_read(drafted, dev(offsets(both)), i32([0] * B), max(both), rows)
        rows, t, s = rows.cpu().numpy(), 0, 0
        for b in range(B):
            seen = np.ones((n[b], both[b]), bool)
            seen[:, length[b]:] = [[m >> j & 1 for j in range(n[b])] for m in trees[b][0]]
            of = rows[s:s + both[b]]
            want, mag, big = lat.attend(q[t:t + n[b]].cpu().numpy().reshape(-1, W), of, of[:, :Dc], np.repeat(seen, Hq, 0), scale)
            # (as in the tests of the attention: an output's and a weight's rounding, the score's, the sums')
            tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -24 * np.abs(of).max() + mag * (
                2.0 ** -11 + 2 * (W + 8) * 2.0 ** -24 * big[:, None] + both[b] * 2.0 ** -26)
            assert (np.abs(o[t:t + n[b]].cpu().numpy().reshape(-1, Dc) - want) <= tol).all()
            t, s = t + n[b], s + both[b]
        # a path from the root is accepted
        paths = []
        for m, (words, depths, parent) in zip(n, trees):
            at, path = int(rng.integers(0, m)), []
            while at >= 0:
                path.insert(0, at)
                at = parent[at]
            paths.append(path)
        k = [len(p) for p in paths]
        us.us_lat_commit(drafted, dev(offsets(k)), i32(sum(paths, [])), pos, 64)
        first = offsets(n)
        kept = x[torch.tensor([int(first[b]) + i for b in range(B) for i in paths[b]], device="cuda")]
        after = [a + b for a, b in zip(length, k)]
        us.us_kv_reserve(pools[1], i32(after))
        us.us_lat_write(chain, r, kept, w, dev(offsets(k)), pos, None, 64)
        length = after
        us.us_kv_reserve(pools[0], i32(length))
        got = []
        for C in (drafted, chain):
            rows = torch.empty(sum(length), W, dtype=torch.float16, device="cuda")
            us.us_lat_read(C, dev(offsets(length)), i32([0] * B), max(length), rows)
            got.append(rows)
        assert torch.equal(*got) and torch.isfinite(got[0]).all()
        assert us.us_get_last_device_status() == us.US_OK
        assert torch.equal(pools[0].held, pools[1].held) and torch.equal(pools[0].free_count, pools[1].free_count)
