"""Attention over the quantised cache where scores are large: weights stay within fp16, and the scores' order stands.

Keys have one direction and different lengths, so that queries of both signs rank them and each row's output is one
stored value (2^-11 of it for its weight, for that weight with V's scale and for the output).  Lengths are apart by
2^-10 and more of themselves, twice a stored scale's step: the next best weight is e^-60 and less from size 250 on."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import dev
from tests.test_gpu_rope import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def us():
    from bitmap_encoded_unstructured_ie_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("elem", ["US_I8", "US_I4"])
@pytest.mark.parametrize("D,G,ctx,n", [(128, 1, 0, 1), (64, 1, 900, 1), (128, 8, 5000, 1), (64, 2, 300, 3), (128, 2, 300, 40), (64, 8, 0, 40), (128, 16, 2000, 9)])
@pytest.mark.parametrize("values", [0.01, 1.0, 400.0])
def test_large_scores(us, elem, D, G, ctx, n, values):
    elem, H, L = getattr(us, elem), 4, ctx + n
    for size in (250, 700, 1000, 2000, 2900, 4000, 5700, 8000, 16000, 23000, 60000):
        rng = np.random.default_rng(size)
        C = us.kv_cache(elem, D, H, 64, -(-L // 64), i32(np.arange(-(-L // 64))[None]))
        along = np.sign(rng.standard_normal(D))
        length = np.concatenate((np.linspace(0.8, 0.9, ctx), 0.95 + 0.05 * (np.arange(n) + 1) / n))
        length[0] = 0.7 if L > 1 else 1.0
        K = np.repeat((size * length[:, None] * along)[:, None], H, 1).astype(np.float16)
        V = (values * rng.standard_normal((L, H, D))).astype(np.float16)
        us.us_kv_write(C, dev(K), dev(V), i32([0, L]), i32([0]), L)
        ko, vo = (torch.empty(L, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
        us.us_kv_read(C, i32([0, L]), i32([0]), L, ko, vo)
        sign = np.where(np.arange(H * G) % 2, -1, 1)
        Q = np.repeat((size * along * sign[:, None])[None], n, 0).astype(np.float16)
        o = torch.empty(n, H * G, D, dtype=torch.float16, device="cuda")
        us.us_attn_kv(C, dev(Q), i32([0, n]), i32([ctx]), None, n, D ** -0.5, o, us.workspace_attn_kv(C, H * G, n))
        assert us.us_get_last_device_status() == us.US_OK
        got, v = o.cpu().numpy().astype(np.float64), vo.cpu().numpy().astype(np.float64)
        for i in range(n):
            best = (0 if i == 0 and ctx == 0 else ctx + i, 0)
            for h in range(H * G):
                want = v[best[h % 2], h // G]
                assert (np.abs(got[i, h] - want) <= 2.0 ** -9 * np.abs(want) + 2.0 ** -23).all(), (size, i, h)
