"""The latent block's example run as a whole: pages, rotation, cache, both forms of the
attention, a captured and replayed graph, against the block's definition in 64 bits.

Tolerance.  What the device rounds to fp16 between the definition's steps: queries,
latent rows, the keys, values or inner queries made of them, the weights, the outputs.
Each is off by 2^-11 of itself, and a sum of products by that of its absolute sum.  With
S the largest sum of |q||k| scale of a row over such absolute sums (keys as
sum |latent||weight|), a score is off by at most 4 2^-11 S, a weight by twice that, and
with A the weighted mean of the values' absolute sums
|err| <= A (4 2^-11 + 8 2^-11 S) + 2^-11."""
import numpy as np
import pytest
import torch

from oracle import lat

pytestmark = pytest.mark.gpu


def test_block_against_its_definition():
    from examples import latent_decode as ex

    seen = []

    def watch(block, x, o, n, pos):
        seen.append((x.cpu().numpy().astype(np.float64), o.cpu().numpy().astype(np.float64), list(n), list(pos)))

    blk, length, y = ex.run(single=20, watch=watch)
    assert length == [37 + 20, 150 + 20, 16 + 20] and blk.pool.held.tolist() == [-(-n // 16) for n in length]
    H, Dn, Dc = blk.H, blk.Dn, blk.Dc
    f = lambda t: t.cpu().numpy().astype(np.float64)  # noqa: E731
    wq, wc, wkv, norm = f(blk.wq), f(blk.wc), f(blk.wkv).reshape(H, 2 * Dn, Dc), f(blk.norm)
    freq = 10000.0 ** (-2.0 * np.arange(32) / 64)
    rows = [np.zeros((0, Dc + 64)) for _ in length]
    worst = 0.0
    for x, o, n, pos in seen:
        t = 0
        for b, k in enumerate(n):
            if not k:
                continue
            xb, p = x[t:t + k], pos[b] + np.arange(k)
            c = xb @ wc.T
            rows[b] = np.concatenate((rows[b], np.concatenate((lat.norm(c[:, :Dc], norm, 1e-6), lat.rotate(c[:, Dc:], p, freq, True)), 1)))
            assert len(rows[b]) == pos[b] + k
            q = (xb @ wq.T).reshape(k, H, Dn + 64)
            q[..., Dn:] = lat.rotate(q[..., Dn:], p, freq, True)
            qa = (np.abs(xb) @ np.abs(wq).T).reshape(k, H, Dn + 64)
            mask = np.tril(np.ones((k, pos[b] + k), bool), pos[b])
            for h in range(H):
                key = np.concatenate((rows[b][:, :Dc] @ wkv[h, :Dn].T, rows[b][:, Dc:]), 1)
                val = rows[b][:, :Dc] @ wkv[h, Dn:].T
                want, _, _ = lat.attend(q[:, h], key, val, mask, blk.scale)
                ka = np.concatenate((np.abs(rows[b][:, :Dc]) @ np.abs(wkv[h, :Dn]).T, np.abs(rows[b][:, Dc:])), 1)
                S = (np.abs(qa[:, h]) @ ka.T * blk.scale).max()
                A = (np.abs(rows[b][:, :Dc]) @ np.abs(wkv[h, Dn:]).T).max()
                err = np.abs(o[t:t + k, h] - want)
                assert (err <= A * (4 + 8 * S) * 2.0 ** -11 + 2.0 ** -11).all()
                worst = max(worst, np.linalg.norm(err) / np.linalg.norm(want))
            t += k
    # (the bound above is of the worst case; roundings are independent, and the whole is off by a few 2^-11)
    assert worst <= 16 * 2.0 ** -11


def test_absorbed_and_expanded_forms_agree():
    """The same tokens as one chunk in the expanded form and one by one in the latent space."""
    from examples import latent_decode as ex

    outs = []
    for prompts, single in (((24, 20, 17), 0), ((23, 19, 16), 1)):
        xs = torch.randn(24 + 20 + 17, 512, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half()
        blk = ex.Block(B=3)
        n = list(prompts)
        us, starts = ex.us, (0, 24, 44)
        x = torch.cat([xs[s:s + k] for s, k in zip(starts, n)])
        us.us_kv_reserve(blk.pool, ex.ints(n))
        y, q, o = blk.chunk(x, ex.offsets(n), ex.ints([0, 0, 0]), max(n), ex.offsets(n), sum(n), max(n))
        last = torch.stack([o[sum(n[:b + 1]) - 1] for b in range(3)])
        if single:
            us.us_kv_reserve(blk.pool, ex.ints([k + 1 for k in n]))
            y, q, last = blk.token(torch.stack([xs[s + k] for s, k in zip(starts, n)]), ex.offsets([1] * 3), ex.ints(n))
        assert us.us_get_last_device_status() == us.US_OK
        outs.append(last.double())
    assert (outs[0] - outs[1]).norm() <= 16 * 2.0 ** -11 * outs[0].norm()
