"""The example of drafted trees, each of its calls against the plain reference.

The reference keeps its own cache: it quantises the projected keys and values,
moves the accepted entries and attends in 64 bits; the device's cache must hold
the same codes and scales after every call.  The attention's tolerance is that of
its own tests: per output 2^-11 |o| + A (2 2^-11 + 2 (D + 8) 2^-24 S) + 2^-24 with
A = sum w|v| / sum w and S the largest sum |q||k| scale.
"""
import importlib.util
import pathlib

import numpy as np
import pytest

from oracle import kv

pytestmark = pytest.mark.gpu
PATH = pathlib.Path(__file__).parent.parent / "examples" / "tree_decode.py"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class Follower:
    def __init__(self, elem):
        self.elem, self.ref, self.calls = elem, None, []

    def __call__(self, blk, pos, paths=None, **call):
        C = blk.cache
        if self.ref is None:
            num_pages, Hkv, page, _ = C.k.shape
            self.ref = kv.Cache(self.elem, blk.D, Hkv, page, num_pages, C.page_table.cpu().numpy())
        if paths is not None:
            for b, path in enumerate(paths):
                self.ref.commit(b, pos[b], path)
            self.same(C, [p + len(path) for p, path in zip(pos, paths)])
            self.calls.append("commit")
            return
        self.forward(blk, pos, **call)

    def same(self, C, length):
        k, v, scale = C.k.cpu().numpy(), C.v.cpu().numpy(), C.scale.cpu().numpy().view(np.float16)
        for b, n in enumerate(length):
            for p in range(n):
                g, s = self.ref.at(b, p)
                for got, want in ((k, self.ref.k), (v, self.ref.v), (scale, self.ref.scale)):
                    assert np.array_equal(got[g, :, s], want[g, :, s]), f"request {b}, position {p}"

    def forward(self, blk, pos, qkv, o, n, parents):
        r, Hq, Hkv = self.ref, blk.Hq, blk.Hkv
        rows, out = qkv.cpu().numpy(), o.cpu().numpy().astype(np.float64)
        t = 0
        for b, k in enumerate(n):
            for i in range(k):
                g, s = r.at(b, pos[b] + i)
                for which, pool in enumerate((r.k, r.v)):
                    x = rows[t + i, Hq + which * Hkv:Hq + (which + 1) * Hkv]
                    c, sc = kv.quantise(x, self.elem)
                    pool[g, :, s], r.scale[g, :, s, which] = kv.pack(c, self.elem), sc
            seen = [[j <= i for j in range(k)] for i in range(k)]
            if parents:
                for i in range(k):
                    line = {i}
                    while parents[b][min(line)] >= 0:                   # a draft's parent comes before it
                        line.add(parents[b][min(line)])
                    seen[i] = [j in line for j in range(k)]
            want, mag, big = kv.attend(r, b, rows[t:t + k, :Hq], pos[b], seen, blk.scale)
            tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -24
                   + mag * (2 * 2.0 ** -11 + 2 * (blk.D + 8) * 2.0 ** -24 * big[..., None]))
            err = np.abs(out[t:t + k] - want)
            assert (err <= tol).all(), f"request {b}: {np.max(err / tol):.2f} times the tolerance"
            t += k
        self.same(blk.cache, [p + k for p, k in zip(pos, n)])
        self.calls.append("tree" if parents else "token" if max(n) == 1 else "prompt")


@pytest.mark.parametrize("elem,D,Hq,Hkv,page", [(kv.I8, 64, 8, 2, 16), (kv.I4, 128, 4, 1, 32)])
def test_prompts_trees_and_single_tokens(example, elem, D, Hq, Hkv, page):
    f = Follower(elem)
    blk, length, y = example.run(steps=2, single=3, watch=f, elem=elem, D=D, Hq=Hq, Hkv=Hkv, page=page)
    assert f.calls == ["prompt"] * 3 + ["tree", "commit"] * 2 + ["token"] * 3
    assert y.shape == (3, blk.hidden) and bool(y.isfinite().all())
